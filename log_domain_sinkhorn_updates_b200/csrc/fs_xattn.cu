// Cross attention on CUDA cores, forward and gradient: every type, head width
// up to 256 and alignment.  fp32 inputs always come here (plain fp32 products,
// like the f32_simt precision of the transport application), and so do bf16
// inputs whose strides or bases a TMA box cannot start on, or with d or dv
// over 128.
//
//   S_ij = scale q_i.k_j + bias_j,  L_i = log sum_j e^{S_ij},  out_i = sum_j e^{S_ij - L_i} v_j
//   D_i = dout_i.out_i,  P = e^{S - L},  dS_ij = P_ij (dout_i.v_j - D_i)
//   dv_j = sum_i P_ij dout_i,  dk_j = scale sum_i dS_ij q_i,  dq_i = scale sum_j dS_ij k_j
//
// Tiles of rows and keys as fp32 in shared memory, 16 x 16 threads with a block
// of each product in registers; where shared memory allows it the next tile
// arrives under this one's arithmetic (fp32: asynchronous copies).  Products go
// two to an instruction (forward, 4 x 1024 x 1024, 8 heads of 64: 348 -> 338 us).
// What bounds it is shared memory's latency: the FMA pipe is 34 to 37 % active,
// the schedulers issue every other cycle (2 x 1024 x 1024, 8 heads of 64: forward
// 25 TFLOP/s, gradient 25).  Where few CTAs stream for long (4 queries of 8 heads
// against 5000 keys: 892 -> 49 us) the gradient's streamed tiles are split into
// parts, whose sums a second kernel adds.  Up to 8 rows a key head (single tokens)
// have a kernel that streams K and V through registers alone: what bounds it is
// the loads that two warps a scheduler keep in flight (fp32, 65536 keys of 8 heads
// of 128: 108 us and the join, 131 back to back; DRAM 61 % of its peak).
//
// The heads that share a key head are rows of one problem: row r = i group + h.
// Keys past the length or masked by the bias are staged as zeros, so nothing
// that stands in their memory reaches a sum.
#include "fs_ops.cuh"

namespace fs {
namespace {

constexpr int kThreads = 128;  // of the joining pass and the row products
constexpr int kTileThreads = 256;
constexpr int kKeys = 64;      // keys of a forward tile
constexpr int kStream = 32;    // streamed rows of a gradient tile
constexpr int kMaxD = 256;
constexpr size_t kMaxSmem = 227 * 1024;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float *o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

// The query of packed row r: r / group without a division (r < 2^31: m = ceil(2^(31 + s) / group), s = ceil(log2
// group), is too large by less than group / group of 2^(31 + s) / r, so the product's integer part is the quotient).
__device__ __forceinline__ int row_query(const AttnParams &p, int r) {
    return p.group == 1 ? r : (int)(__umulhi((unsigned)r, p.group_mul) >> p.group_shift);
}
// Element offset of packed row r (of key head c, problem b) in a query-side tensor.
__device__ __forceinline__ long long row_off(const fs_view &s, const AttnParams &p, int b, int c, int r) {
    const int i = row_query(p, r);
    return s.batch * b + s.token * i + s.head * (c * p.group + r - i * p.group);
}
__device__ __forceinline__ size_t row_stat(const AttnParams &p, int b, int c, int r) {
    const int i = row_query(p, r);
    return ((size_t)b * p.heads + c * p.group + r - i * p.group) * p.n + i;
}

// Row stride in shared memory of a tile of width w: an odd number of 16-byte pieces, so that eight rows' pieces at
// one column lie in different banks.
__host__ __device__ inline int smem_stride(int w) { return ((w + 3) / 4 | 1) * 4; }
// The tiles' stride in a kernel of C 64-column pieces: known to the compiler, so that rows are offsets of one address,
// but for the widest, whose shared memory it would cost.
template <int C>
__host__ __device__ __forceinline__ int tile_stride(int w) {
    return C <= 2 ? 64 * C + 4 : smem_stride(w);
}

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}
// `cnt` rows of width w into sm (stride ld, zeros up to a multiple of 4); row(r) is a row's address, or
// null for a row of zeros.  vec: every row is aligned to four elements.
template <class T, class Row>
__device__ void stage(float *sm, int ld, int cnt, int w, bool vec, Row row) {
    const int pieces = (w + 3) / 4;
    int per = 1;
    while (per < pieces) per *= 2;
    const int k = (int)threadIdx.x % per * 4, step = kTileThreads / per;
    for (int r0 = (int)threadIdx.x / per; r0 < cnt; r0 += 4 * step) {
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = r0 + u * step;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r >= cnt || k >= w) continue;
            const T *p = row(r);
            if (!p) continue;
            if (vec && k + 4 <= w) {
                v[u] = load4(p + k);
            } else {
                v[u].x = to_f(p[k]);
                if (k + 1 < w) v[u].y = to_f(p[k + 1]);
                if (k + 2 < w) v[u].z = to_f(p[k + 2]);
                if (k + 3 < w) v[u].w = to_f(p[k + 3]);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (r0 + u * step < cnt && k < w) *reinterpret_cast<float4 *>(sm + (r0 + u * step) * ld + k) = v[u];
    }
}
// The same by asynchronous copies where that can be (fp32, aligned rows); the caller commits and waits.
template <class T, class Row>
__device__ void stage_tile(float *sm, int ld, int cnt, int w, bool vec, const T *any, Row row) {
    if (sizeof(T) != 4 || !vec) {
        stage<T>(sm, ld, cnt, w, vec, row);
        return;
    }
    const int pieces = (w + 3) / 4;
    int per = 1;
    while (per < pieces) per *= 2;
    const int k = (int)threadIdx.x % per * 4, step = kTileThreads / per;
    if (k >= w) return;
    for (int r = (int)threadIdx.x / per; r < cnt; r += step) {
        const T *src = row(r);
        const int bytes = src ? min(16, (w - k) * 4) : 0;  // the rest of the piece becomes zeros
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(sm + r * ld + k));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src ? src + k : any), "r"(bytes)
                     : "memory");
    }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// packed query rows [r0, ...), and keys [j0, ...) of a problem (zeros where a key is masked, or not below j_end)
template <class T>
__device__ void stage_rows(float *sm, int ld, const void *src, const fs_view &s, const AttnParams &p, int b, int c, int r0,
                           int cnt, int w, bool vec) {
    const int rows = p.n * p.group;
    stage_tile<T>(sm, ld, cnt, w, vec, (const T *)src, [&](int r) -> const T * {
        return r0 + r < rows ? (const T *)src + row_off(s, p, b, c, r0 + r) : nullptr;
    });
}
template <class T>
__device__ void stage_keys(float *sm, int ld, const void *src, const fs_view &s, const AttnParams &p, int b, int c, int j0,
                           int cnt, int w, int j_end, bool vec) {
    const T *base = (const T *)src + s.batch * b + s.head * c;
    stage_tile<T>(sm, ld, cnt, w, vec, (const T *)src, [&](int j) -> const T * {
        return attn_masked(p, b, j0 + j, j_end) ? nullptr : base + s.token * (j0 + j);
    });
}

// acc[u][w] = sum_k a[u][k] b[BSTEP w][k] over rows of the tiles (strides la and lb); even and odd k are summed apart
// and added at the end.
template <int U, int W, int BSTEP>
__device__ __forceinline__ void dots(float (&acc)[U][W], const float *a, int la, const float *b, int lb, int width) {
    uint64_t two[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int w = 0; w < W; ++w) two[u][w] = 0ull;
    for (int k = 0; k < width; k += 4) {
        ulonglong2 x[U], y[W];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = *reinterpret_cast<const ulonglong2 *>(a + u * la + k);
#pragma unroll
        for (int w = 0; w < W; ++w) y[w] = *reinterpret_cast<const ulonglong2 *>(b + w * BSTEP * lb + k);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int w = 0; w < W; ++w)
                two[u][w] = fma2(x[u].y, y[w].y, fma2(x[u].x, y[w].x, two[u][w]));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float even, odd;
            unpack2(two[u][w], even, odd);
            acc[u][w] = even + odd;
        }
}
// o[u][k] += sum_j wt[u][j] val[j][col + 64 k .. + 3] over `cnt` rows of val
template <int U, int C>
__device__ __forceinline__ void weigh(float4 (&o)[U][C], const float *wt, int lw, const float *val, int lv, int cnt,
                                      int col, int width) {
    for (int j = 0; j < cnt; j += 4) {
        float4 f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) f[u] = *reinterpret_cast<const float4 *>(wt + u * lw + j);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            if (col + 64 * k >= width) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = *reinterpret_cast<const float4 *>(val + (j + i) * lv + col + 64 * k);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float g = i == 0 ? f[u].x : i == 1 ? f[u].y : i == 2 ? f[u].z : f[u].w;
                    o[u][k].x = fmaf(g, v.x, o[u][k].x);
                    o[u][k].y = fmaf(g, v.y, o[u][k].y);
                    o[u][k].z = fmaf(g, v.z, o[u][k].z);
                    o[u][k].w = fmaf(g, v.w, o[u][k].w);
                }
            }
        }
    }
}
template <class T>
__device__ __forceinline__ void put4(T *dst, float4 v, int k, int width, float mul) {
    if (k < width) from_f(v.x * mul, dst + k);
    if (k + 1 < width) from_f(v.y * mul, dst + k + 1);
    if (k + 2 < width) from_f(v.z * mul, dst + k + 2);
    if (k + 3 < width) from_f(v.w * mul, dst + k + 3);
}

// One CTA: 16 RPT packed rows of a key head over one part of the keys, 16 x 16 threads of RPT rows x 4 keys.  C:
// 64-column pieces of the widths.
template <class T, int RPT, int C>
__global__ void __launch_bounds__(kTileThreads) xattn_simt_kernel(const AttnParams p, bool vec, int bufs) {
    extern __shared__ __align__(16) float sm[];
    constexpr int R = 16 * RPT, LP = kKeys + 4;
    const AttnUnit unit = p.k_len ? attn_unit<true>(p) : attn_unit<false>(p);
    const int r0 = unit.r0, c = unit.c, b = unit.b, j_beg = unit.j_beg, j_end = unit.j_end;
    const int ld = tile_stride<C>(p.d), lv = tile_stride<C>(p.dv);
    const int tile = kKeys * (ld + lv) + kKeys;  // K, V and the bias of one buffer
    float *sTop = sm, *sQ = sm + 4, *sP = sQ + R * ld, *ring = sP + R * LP;
    const float top = attn_top<kTileThreads>(p, b, j_beg, j_end, sP);
    if (attn_stats_done(p, unit, top)) return;
    if (threadIdx.x == 0) *sTop = top;  // read again at the end
    __syncthreads();
    // tile t into buffer t % bufs: with two, it arrives under the arithmetic of the tile before
    auto fetch = [&](int t) {
        float *sK = ring + (bufs == 2 ? t & 1 : 0) * tile, *sV = sK + kKeys * ld, *sB = sV + kKeys * lv;
        const int j0 = j_beg + t * kKeys;
        if (threadIdx.x < kKeys) sB[threadIdx.x] = attn_bias2(p, b, j0 + threadIdx.x, j_end, top);
        stage_keys<T>(sK, ld, p.k, p.ks, p, b, c, j0, kKeys, p.d, j_end, vec);
        stage_keys<T>(sV, lv, p.v, p.vs, p, b, c, j0, kKeys, p.dv, j_end, vec);
    };
    const int nt = j_end > j_beg && top != -INFINITY ? (j_end - j_beg + kKeys - 1) / kKeys : 0;
    stage_rows<T>(sQ, ld, p.q, p.qs, p, b, c, r0, R, p.d, vec);
    if (bufs == 2 && nt > 0) fetch(0);
    stage_commit();
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float4 o[RPT][C];
    float mx[RPT], l[RPT];
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        mx[u] = -INFINITY;
        l[u] = 0.f;
#pragma unroll
        for (int k = 0; k < C; ++k) o[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int t = 0; t < nt; ++t) {
        if (bufs == 1) {
            __syncthreads();
            fetch(t);
            stage_commit();
            stage_wait<0>();
        } else {
            if (t + 1 < nt) fetch(t + 1);
            stage_commit();
            stage_wait<1>();
        }
        __syncthreads();
        const float *sK = ring + (bufs == 2 ? t & 1 : 0) * tile, *sV = sK + kKeys * ld, *sB = sV + kKeys * lv;
        float z[RPT][4];
        dots<RPT, 4, 16>(z, sQ + ti * RPT * ld, ld, sK + tj * ld, ld, p.d);
#pragma unroll
        for (int u = 0; u < RPT; ++u) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                z[u][w] = fmaf(z[u][w], p.scale2, sB[tj + 16 * w]);
                top = fmaxf(top, z[u][w]);
            }
            for (int w = 8; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
            const float mn = fmaxf(mx[u], top);
            const float ref = mn == -INFINITY ? 0.f : mn;  // nothing but masked keys so far: every term below is 0
            const float cor = exp2f(mx[u] - ref);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float e = exp2f(z[u][w] - ref);
                sP[(ti * RPT + u) * LP + tj + 16 * w] = e;
                sum += e;
            }
            for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
            l[u] = l[u] * cor + sum;
            mx[u] = mn;
#pragma unroll
            for (int k = 0; k < C; ++k) {
                o[u][k].x *= cor;
                o[u][k].y *= cor;
                o[u][k].z *= cor;
                o[u][k].w *= cor;
            }
        }
        __syncwarp();  // a row's weights are written and read by its 16 threads, of one warp
        weigh<RPT, C>(o, sP + ti * RPT * LP, LP, sV, lv, kKeys, 4 * tj, p.dv);
        if (bufs == 2) __syncthreads();  // the buffer is filled again
    }
    stage_wait<0>();
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int r = r0 + ti * RPT + u;
        if (r >= p.n * p.group) continue;
        if (!unit.whole) {
            const size_t at = unit.part + ti * RPT + u;
            if (tj == 0) p.part_ml[at] = {*sTop, mx[u], l[u]};
#pragma unroll
            for (int k = 0; k < C; ++k) put4(p.part_o + at * p.dv, o[u][k], 4 * tj + 64 * k, p.dv, 1.f);
            continue;
        }
        const float inv = l[u] == 0.f ? 0.f : 1.f / l[u];  // 0: no key is left (a NaN row stays NaN)
        if (p.stats) {
            if (tj == 0) p.lse2[row_stat(p, b, c, r)] = (float)((double)mx[u] + log2((double)l[u]));
            continue;
        }
        T *dst = (T *)p.out + row_off(p.os, p, b, c, r);
#pragma unroll
        for (int k = 0; k < C; ++k) put4(dst, o[u][k], 4 * tj + 64 * k, p.dv, inv);
        if (p.lse && tj == 0)
            p.lse[row_stat(p, b, c, r)] =
                l[u] == 0.f ? -INFINITY : (float)(((double)mx[u] + log2((double)l[u])) * kLn2d + *sTop);
    }
}

// Few rows (a unit of RT <= 4): what counts is to stream K and V.  Eight lanes take a key (four keys a warp at once),
// each lane a 16-byte piece in every 32 of the width, so that a row is read in whole lines and a score takes three
// shuffles; every group of lanes keeps its own running maximum, sum and output, joined at the end (lanes by shuffles,
// warps through shared memory, in a fixed order).  The next keys' rows are loaded before this one's arithmetic.  C:
// 32-element pieces of the widths.
template <class T, int RT, int C>
__global__ void __launch_bounds__(kTileThreads, 1) xattn_token_kernel(const AttnParams p) {
    __shared__ float so[8][RT][32 * C + 4];
    __shared__ float2 sml[8][RT];
    const AttnUnit unit = p.k_len ? attn_unit<true>(p) : attn_unit<false>(p);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, grp = lane / 8, sub = lane % 8;
    const int b = unit.b, c = unit.c, rows = p.n * p.group;
    const float bias_top = attn_top<kTileThreads>(p, b, unit.j_beg, unit.j_end, &sml[0][0].x);
    const int j_end = bias_top == -INFINITY ? unit.j_beg : unit.j_end;
    float4 q[RT][C], o[RT][C];
    float mx[RT], l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        mx[r] = -INFINITY;
        l[r] = 0.f;
        const bool live = unit.r0 + r < rows;
        const T *src = (const T *)p.q + (live ? row_off(p.qs, p, b, c, unit.r0 + r) : 0);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int e = 32 * k + 4 * sub;
            q[r][k] = live && e < p.d ? load4(src + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            q[r][k].x *= p.scale2, q[r][k].y *= p.scale2, q[r][k].z *= p.scale2, q[r][k].w *= p.scale2;
            o[r][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    const T *kb = (const T *)p.k + p.ks.batch * b + p.ks.head * c;
    const T *vb = (const T *)p.v + p.vs.batch * b + p.vs.head * c;
    float4 kn[C], vn[C];
    float bn;
    auto fetch = [&](int j) {  // key j's bias, and its rows unless it is masked (or past the part)
        bn = attn_bias2(p, b, j, j_end, bias_top);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int e = 32 * k + 4 * sub;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            kn[k] = bn != -INFINITY && e < p.d ? load4(kb + p.ks.token * j + e) : zero;
            vn[k] = bn != -INFINITY && e < p.dv ? load4(vb + p.vs.token * j + e) : zero;
        }
    };
    const int first = unit.j_beg + 4 * warp + grp;
    fetch(first);
    for (int j = first; j - grp < j_end; j += 32) {  // whole warps: the shuffles take every lane
        float4 kc[C], vc[C];
        const float bias = bn;
#pragma unroll
        for (int k = 0; k < C; ++k) kc[k] = kn[k], vc[k] = vn[k];
        fetch(j + 32);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float z = 0.f;
#pragma unroll
            for (int k = 0; k < C; ++k)
                z = fmaf(q[r][k].x, kc[k].x,
                         fmaf(q[r][k].y, kc[k].y, fmaf(q[r][k].z, kc[k].z, fmaf(q[r][k].w, kc[k].w, z))));
            z += __shfl_xor_sync(~0u, z, 1);
            z += __shfl_xor_sync(~0u, z, 2);
            z += __shfl_xor_sync(~0u, z, 4);
            z += bias;
            if (z > mx[r]) {  // the same on the eight lanes of the key
                const float f = exp2f(mx[r] - z);
                mx[r] = z;
                l[r] *= f;
#pragma unroll
                for (int k = 0; k < C; ++k) o[r][k].x *= f, o[r][k].y *= f, o[r][k].z *= f, o[r][k].w *= f;
            }
            const float e = z == -INFINITY ? 0.f : exp2f(z - mx[r]);  // a NaN stays one
            l[r] += e;
#pragma unroll
            for (int k = 0; k < C; ++k) {
                o[r][k].x = fmaf(e, vc[k].x, o[r][k].x);
                o[r][k].y = fmaf(e, vc[k].y, o[r][k].y);
                o[r][k].z = fmaf(e, vc[k].z, o[r][k].z);
                o[r][k].w = fmaf(e, vc[k].w, o[r][k].w);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        float top = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 8));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
        const float f = exp2f(mx[r] - (top == -INFINITY ? 0.f : top));
        float lw = l[r] * f;
        lw += __shfl_xor_sync(~0u, lw, 8);
        lw += __shfl_xor_sync(~0u, lw, 16);
        if (lane == 0) sml[warp][r] = make_float2(top, lw);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            float4 x = o[r][k];
            x.x *= f, x.y *= f, x.z *= f, x.w *= f;
#pragma unroll
            for (int s = 8; s <= 16; s *= 2) {
                x.x += __shfl_xor_sync(~0u, x.x, s);
                x.y += __shfl_xor_sync(~0u, x.y, s);
                x.z += __shfl_xor_sync(~0u, x.z, s);
                x.w += __shfl_xor_sync(~0u, x.w, s);
            }
            if (grp == 0) *reinterpret_cast<float4 *>(&so[warp][r][32 * k + 4 * sub]) = x;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < RT * p.dv; e += kTileThreads) {
        const int r = e / p.dv, k = e % p.dv, row = unit.r0 + r;
        if (row >= rows) break;  // rows come in order
        float top = -INFINITY, sum = 0.f, x = 0.f;
        for (int w = 0; w < 8; ++w) top = fmaxf(top, sml[w][r].x);
        const float ref = top == -INFINITY ? 0.f : top;
        for (int w = 0; w < 8; ++w) {
            const float f = exp2f(sml[w][r].x - ref);
            sum += sml[w][r].y * f;
            x = fmaf(so[w][r][k], f, x);
        }
        if (!unit.whole) {
            if (k == 0) p.part_ml[unit.part + r] = {bias_top, top, sum};
            p.part_o[(unit.part + r) * p.dv + k] = x;
        } else {
            from_f(sum == 0.f ? 0.f : x / sum, (T *)p.out + row_off(p.os, p, b, c, row) + k);
            if (p.lse && k == 0)
                p.lse[row_stat(p, b, c, row)] =
                    sum == 0.f ? -INFINITY : (float)(((double)top + log2((double)sum)) * kLn2d + bias_top);
        }
    }
}

// Joins the parts of a row, in the parts' order.  One warp per packed row.
template <class T>
__global__ void __launch_bounds__(kThreads) xattn_combine_kernel(const AttnParams p) {
    const size_t all = (size_t)p.tail_units * p.unit_rows;
    const size_t at = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (at >= all) return;
    const int lane = threadIdx.x % 32;
    const int unit = p.main_units + (int)(at / p.unit_rows);
    const int r = unit % p.blocks * p.unit_rows + (int)(at % p.unit_rows);
    const int c = unit / p.blocks % p.kv_heads, place = unit / p.blocks / p.kv_heads;
    const int b = p.k_len ? attn_problem<true>(p, place) : place;
    if (r >= p.n * p.group) return;
    grid_dependency_wait();
    // a lane's parts, one in every 32
    AttnPart ml[kAttnParts / 32];
#pragma unroll
    for (int c32 = 0; c32 < kAttnParts / 32; ++c32) {
        ml[c32] = AttnPart{0.f, -INFINITY, 0.f};
        if (32 * c32 < p.splits && 32 * c32 + lane < p.splits) ml[c32] = p.part_ml[(32 * c32 + lane) * all + at];
    }
    // the largest bias reference (of parts with a key), and the largest score reference measured from it
    float from = 0.f, mx = -INFINITY;
    if (p.bias) {
        from = -INFINITY;
#pragma unroll
        for (int c32 = 0; c32 < kAttnParts / 32; ++c32)
            if (ml[c32].l != 0.f) from = fmaxf(from, ml[c32].top);
        for (int w = 16; w; w >>= 1) from = fmaxf(from, __shfl_xor_sync(~0u, from, w));
    }
#pragma unroll
    for (int c32 = 0; c32 < kAttnParts / 32; ++c32) {
        if (ml[c32].l != 0.f) ml[c32].m += (ml[c32].top - from) * kLog2e;
        mx = fmaxf(mx, ml[c32].m);
    }
    for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float l = 0.f, o[kMaxD / 32];
#pragma unroll
    for (int k = 0; k < kMaxD / 32; ++k) o[k] = 0.f;
#pragma unroll
    for (int c32 = 0; c32 < kAttnParts / 32; ++c32) {
        const int s0 = 32 * c32;
        if (s0 >= p.splits) break;
        // a lane's part: its weight; 0 where it has no key (its sums were not written)
        const float f = ml[c32].l == 0.f ? 0.f : exp2f(ml[c32].m - ref);
        const unsigned has = __ballot_sync(~0u, ml[c32].l != 0.f);
        float lw = ml[c32].l * f;
        for (int w = 16; w; w >>= 1) lw += __shfl_xor_sync(~0u, lw, w);
        l += lw;
        const int cnt = min(32, p.splits - s0);
        if (p.dv % 4 == 0 && p.dv <= 128) {
            // four consecutive values a lane, kept in o[0..3]
            for (int j = 0; j < cnt; j += 4) {
                float4 v[4];
                float fj[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    fj[u] = __shfl_sync(~0u, f, (j + u) & 31);
                    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (j + u < cnt && (has >> (j + u) & 1u) && 4 * lane < p.dv)
                        v[u] = *reinterpret_cast<const float4 *>(p.part_o + ((s0 + j + u) * all + at) * p.dv + 4 * lane);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    o[0] = fmaf(v[u].x, fj[u], o[0]);
                    o[1] = fmaf(v[u].y, fj[u], o[1]);
                    o[2] = fmaf(v[u].z, fj[u], o[2]);
                    o[3] = fmaf(v[u].w, fj[u], o[3]);
                }
            }
        } else {
            for (int j = 0; j < cnt; ++j) {
                const float fj = __shfl_sync(~0u, f, j);
                if (!(has >> j & 1u)) continue;
#pragma unroll
                for (int k = 0; k < kMaxD / 32; ++k)
                    if (lane + 32 * k < p.dv) o[k] = fmaf(p.part_o[((s0 + j) * all + at) * p.dv + lane + 32 * k], fj, o[k]);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: no key is left (a NaN row stays NaN)
    T *dst = (T *)p.out + row_off(p.os, p, b, c, r);
    const bool four = p.dv % 4 == 0 && p.dv <= 128;
#pragma unroll
    for (int k = 0; k < kMaxD / 32; ++k) {
        const int e = four ? (k < 4 ? 4 * lane + k : p.dv) : lane + 32 * k;
        if (e < p.dv) from_f(o[k] * inv, dst + e);
    }
    if (p.lse && lane == 0)
        p.lse[row_stat(p, b, c, r)] = l == 0.f ? -INFINITY : (float)(((double)mx + log2((double)l)) * kLn2d + from);
}

// D_i = dout_i.out_i of every (query, head) of a problem: `per` lanes take a row, eight elements each at a time.  out is
// the stored one, in bf16 off by 2^-8 at most: a gradient then needs no fp32 copy of it.  And
// its base-2 LSE, unless the forward kernels have taken that (AttnParams::stats).
template <class T>
__global__ void __launch_bounds__(kThreads) xattn_dot_kernel(const AttnParams p, int per, bool vec) {
    const unsigned at = (blockIdx.x * kThreads + threadIdx.x) / (unsigned)per, rows = (unsigned)(p.n * p.heads);
    const int sub = threadIdx.x % per, b = blockIdx.y;
    const bool live = at < rows;
    const int h = (int)(at % (unsigned)p.heads), i = (int)(at / (unsigned)p.heads);
    const size_t to = ((size_t)b * p.heads + h) * p.n + i;
    const float lse = live && sub == 0 ? p.lse[to] : 0.f;
    float s = 0.f;
    if (live) {
        const T *o = (const T *)p.out + p.os.batch * b + p.os.token * i + p.os.head * h;
        const T *g = (const T *)p.dout + p.dos.batch * b + p.dos.token * i + p.dos.head * h;
        for (int k = 8 * sub; k < p.dv; k += 8 * per) {
            if (vec && k + 8 <= p.dv) {
                const float4 x0 = load4(o + k), x1 = load4(o + k + 4), y0 = load4(g + k), y1 = load4(g + k + 4);
                s = fmaf(x0.x, y0.x, fmaf(x0.y, y0.y, fmaf(x0.z, y0.z, fmaf(x0.w, y0.w, s))));
                s = fmaf(x1.x, y1.x, fmaf(x1.y, y1.y, fmaf(x1.z, y1.z, fmaf(x1.w, y1.w, s))));
            } else {
                for (int u = k; u < min(k + 8, p.dv); ++u) s = fmaf(to_f(o[u]), to_f(g[u]), s);
            }
        }
    }
    for (int w = per / 2; w; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
    grid_dependency_wait();
    if (!live || sub) return;
    p.dot[to] = s;
    if (!p.top || p.top[b] == 0.f || p.top[b] == -INFINITY) p.lse2[to] = lse * kLog2e;
}

// KEYS: one CTA keeps 16 U keys of a key head (K, V) and streams its packed rows (Q, dO) in tiles of 32: dk and dv.
// Otherwise: 16 U packed rows (Q, dO) against streamed keys (K, V): dq.  16 x 16 threads: U kept rows x 2 streamed
// ones of the scores, U kept rows x 4 columns a piece of the sums.
template <class T, bool KEYS, int U, int C>
__device__ void grad_pass(const AttnParams &p, bool vec, int bufs, int block, int part, float *sm) {
    constexpr int LS = kStream + 4, kKept = 16 * U;
    const int c = blockIdx.y % p.kv_heads, b = blockIdx.y / p.kv_heads, t0 = block * kKept;
    const int ld = tile_stride<C>(p.d), lv = tile_stride<C>(p.dv);
    float *a1 = sm, *a2 = a1 + kKept * ld, *sP = a2 + kKept * lv, *sS = sP + kKept * LS;
    float *kb = sS + kKept * LS, *kd = kb + kKept;  // kept: bias, or base-2 LSE and D
    float *ring = kd + kKept;
    const int tile = kStream * (ld + lv) + 2 * kStream;  // the streamed pair, and bias, or base-2 LSE and D
    const int keys = attn_grad_keys(p, b), rows = p.n * p.group;
    const float top = p.top ? p.top[b] : 0.f;
    const int all = ((KEYS ? (t0 < keys ? rows : 0) : keys) + kStream - 1) / kStream;
    const int parts = KEYS ? p.key_parts : p.row_parts;
    const int t_beg = (int)((long long)all * part / parts), nt = (int)((long long)all * (part + 1) / parts) - t_beg;
    // base-2 LSE (+inf: an empty row, or one past the end) and D of packed row r
    auto stat = [&](int r, float *lse2, float *d) {
        *lse2 = INFINITY;
        *d = 0.f;
        if (r < rows) {
            const float v = p.lse2[row_stat(p, b, c, r)];
            if (v != -INFINITY) *lse2 = v;
            *d = p.dot[row_stat(p, b, c, r)];
        }
    };
    if (threadIdx.x < kKept) {
        if (KEYS)
            kb[threadIdx.x] = attn_bias2(p, b, t0 + threadIdx.x, keys, top);
        else
            stat(t0 + threadIdx.x, kb + threadIdx.x, kd + threadIdx.x);
    }
    auto fetch = [&](int t) {  // as in the forward
        float *b1 = ring + (bufs == 2 ? t & 1 : 0) * tile, *b2 = b1 + kStream * ld, *sb = b2 + kStream * lv, *sd = sb + kStream;
        const int u0 = (t_beg + t) * kStream;
        if (threadIdx.x < kStream) {
            if (KEYS)
                stat(u0 + threadIdx.x, sb + threadIdx.x, sd + threadIdx.x);
            else
                sb[threadIdx.x] = attn_bias2(p, b, u0 + threadIdx.x, keys, top);
        }
        if (KEYS) {
            stage_rows<T>(b1, ld, p.q, p.qs, p, b, c, u0, kStream, p.d, vec);
            stage_rows<T>(b2, lv, p.dout, p.dos, p, b, c, u0, kStream, p.dv, vec);
        } else {
            stage_keys<T>(b1, ld, p.k, p.ks, p, b, c, u0, kStream, p.d, keys, vec);
            stage_keys<T>(b2, lv, p.v, p.vs, p, b, c, u0, kStream, p.dv, keys, vec);
        }
    };
    if (KEYS) {
        stage_keys<T>(a1, ld, p.k, p.ks, p, b, c, t0, kKept, p.d, keys, vec);
        stage_keys<T>(a2, lv, p.v, p.vs, p, b, c, t0, kKept, p.dv, keys, vec);
    } else {
        stage_rows<T>(a1, ld, p.q, p.qs, p, b, c, t0, kKept, p.d, vec);
        stage_rows<T>(a2, lv, p.dout, p.dos, p, b, c, t0, kKept, p.dv, vec);
    }
    if (bufs == 2 && nt > 0) fetch(0);
    stage_commit();
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float4 g1[U][C], g2[U][KEYS ? C : 1];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < C; ++k) {
            g1[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (KEYS) g2[u][KEYS ? k : 0] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    for (int t = 0; t < nt; ++t) {
        if (bufs == 1) {
            __syncthreads();
            fetch(t);
            stage_commit();
            stage_wait<0>();
        } else {
            if (t + 1 < nt) fetch(t + 1);
            stage_commit();
            stage_wait<1>();
        }
        __syncthreads();
        const float *b1 = ring + (bufs == 2 ? t & 1 : 0) * tile, *b2 = b1 + kStream * ld;
        const float *sb = b2 + kStream * lv, *sd = sb + kStream;
        float s[U][2], g[U][2];
        dots<U, 2, 16>(s, a1 + ti * U * ld, ld, b1 + tj * ld, ld, p.d);
        dots<U, 2, 16>(g, a2 + ti * U * lv, lv, b2 + tj * lv, lv, p.dv);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int kept = ti * U + u, str = tj + 16 * w;
                const float bias = KEYS ? kb[kept] : sb[str], lse2 = KEYS ? sb[str] : kb[kept];
                const float dd = KEYS ? sd[str] : kd[kept];
                const bool off = bias == -INFINITY || lse2 == INFINITY;
                const float pr = off ? 0.f : exp2f(fmaf(s[u][w], p.scale2, bias) - lse2);
                if (KEYS) sP[kept * LS + str] = pr;
                sS[kept * LS + str] = off ? 0.f : pr * (g[u][w] - dd);
            }
        __syncwarp();  // a kept row's weights are written and read by its 16 threads, of one warp
        weigh<U, C>(g1, sS + ti * U * LS, LS, b1, ld, kStream, 4 * tj, p.d);
        if constexpr (KEYS) weigh<U, C>(g2, sP + ti * U * LS, LS, b2, lv, kStream, 4 * tj, p.dv);
        if (bufs == 2) __syncthreads();  // the buffer is filled again
    }
    stage_wait<0>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = t0 + ti * U + u;
        if (at >= (KEYS ? p.m : rows)) continue;
        if (KEYS && kb[ti * U + u] == -INFINITY) {  // takes no part: zeros, whatever stands in a query or its gradient
#pragma unroll
            for (int k = 0; k < C; ++k) g1[u][k] = g2[u][KEYS ? k : 0] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (parts > 1) {  // a part: its raw sums
            const int blocks = ((KEYS ? p.m : rows) + kKept - 1) / kKept;
            const size_t to = ((size_t)part * gridDim.y + blockIdx.y) * blocks * kKept + at;
            float *d1 = (KEYS ? p.part_dk : p.part_dq) + to * p.d;
#pragma unroll
            for (int k = 0; k < C; ++k) put4(d1, g1[u][k], 4 * tj + 64 * k, p.d, 1.f);
            if (KEYS) {
                float *d2 = p.part_dv + to * p.dv;
#pragma unroll
                for (int k = 0; k < C; ++k) put4(d2, g2[u][KEYS ? k : 0], 4 * tj + 64 * k, p.dv, 1.f);
            }
            continue;
        }
        T *d1 = KEYS ? (T *)p.dk + p.dks.batch * b + p.dks.token * at + p.dks.head * c
                     : (T *)p.dq + row_off(p.dqs, p, b, c, at);
#pragma unroll
        for (int k = 0; k < C; ++k) put4(d1, g1[u][k], 4 * tj + 64 * k, p.d, p.scale);
        if (KEYS) {
            T *d2 = (T *)p.dv_out + p.dvs.batch * b + p.dvs.token * at + p.dvs.head * c;
#pragma unroll
            for (int k = 0; k < C; ++k) put4(d2, g2[u][KEYS ? k : 0], 4 * tj + 64 * k, p.dv, 1.f);
        }
    }
}

// Both passes in one launch: key_blocks CTAs of the first, then those of the second.
template <class T, int U, int C>
__global__ void __launch_bounds__(kTileThreads)
    xattn_grad_kernel(const AttnParams p, bool vec, int bufs, int key_blocks) {
    extern __shared__ __align__(16) float sm[];
    const int x = blockIdx.x, keys = key_blocks * p.key_parts;
    if (x < keys)
        grad_pass<T, true, U, C>(p, vec, bufs, x / p.key_parts, x % p.key_parts, sm);
    else
        grad_pass<T, false, U, C>(p, vec, bufs, (x - keys) / p.row_parts, (x - keys) % p.row_parts, sm);
}

// Adds the parts' sums in their order, an element a thread: dk and dv of every key, then dq of every row.
template <class T>
__global__ void __launch_bounds__(256) xattn_grad_join_simt_kernel(const AttnParams p, int key_padded, int row_padded) {
    const int hb = blockIdx.y, c = hb % p.kv_heads, b = hb / p.kv_heads, rows = p.n * p.group, wide = p.d + p.dv;
    const size_t keys = p.key_parts > 1 ? (size_t)p.m * wide : 0, e = (size_t)blockIdx.x * 256 + threadIdx.x;
    grid_dependency_wait();
    const float *src;
    T *dst;
    size_t step;
    int parts;
    float mul = p.scale;
    if (e < keys) {
        const int row = (int)(e / wide), k = (int)(e % wide), width = k < p.d ? p.d : p.dv, col = k < p.d ? k : k - p.d;
        const fs_view &s = k < p.d ? p.dks : p.dvs;
        if (k >= p.d) mul = 1.f;
        src = (k < p.d ? p.part_dk : p.part_dv) + ((size_t)hb * key_padded + row) * width + col;
        dst = (T *)(k < p.d ? p.dk : p.dv_out) + s.batch * b + s.token * row + s.head * c + col;
        step = (size_t)gridDim.y * key_padded * width;
        parts = p.key_parts;
    } else {
        if (p.row_parts == 1 || e - keys >= (size_t)rows * p.d) return;
        const int row = (int)((e - keys) / p.d), col = (int)((e - keys) % p.d);
        src = p.part_dq + ((size_t)hb * row_padded + row) * p.d + col;
        dst = (T *)p.dq + row_off(p.dqs, p, b, c, row) + col;
        step = (size_t)gridDim.y * row_padded * p.d;
        parts = p.row_parts;
    }
    float x = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) x += src[i * step];
    from_f(x * mul, dst);
}

// Whether four elements of every row can be loaded at once.
template <class T>
bool aligned4(const void *base, const fs_view &s) {
    return reinterpret_cast<uintptr_t>(base) % (4 * sizeof(T)) == 0 && s.batch % 4 == 0 && s.token % 4 == 0 &&
           s.head % 4 == 0;
}

template <class T, int RPT, int C>
cudaError_t fwd(const AttnParams &p, cudaStream_t s) {
    constexpr int R = 16 * RPT;
    const int ld = tile_stride<C>(p.d), lv = tile_stride<C>(p.dv);
    const size_t fixed = 4 + (size_t)R * ld + R * (kKeys + 4);
    const size_t tile = (size_t)kKeys * (ld + lv) + kKeys;
    const int bufs = (fixed + 2 * tile) * sizeof(float) <= kMaxSmem ? 2 : 1;
    const size_t smem = (fixed + bufs * tile) * sizeof(float);
    cudaError_t e = allow_smem<&xattn_simt_kernel<T, RPT, C>>(smem);
    if (e != cudaSuccess) return e;
    const bool vec = aligned4<T>(p.q, p.qs) && aligned4<T>(p.k, p.ks) && aligned4<T>(p.v, p.vs);
    xattn_simt_kernel<T, RPT, C><<<p.main_units + p.tail_units * p.splits, kTileThreads, smem, s>>>(p, vec, bufs);
    return cudaGetLastError();
}
template <class T, int RPT>
cudaError_t fwd_width(const AttnParams &p, cudaStream_t s) {
    const int w = p.d > p.dv ? p.d : p.dv;
    return w <= 64 ? fwd<T, RPT, 1>(p, s) : w <= 128 ? fwd<T, RPT, 2>(p, s) : fwd<T, RPT, 4>(p, s);
}
template <class T, int RT>
cudaError_t token(const AttnParams &p, cudaStream_t s) {
    const int ctas = p.main_units + p.tail_units * p.splits, w = p.d > p.dv ? p.d : p.dv;
    if (w <= 32)
        xattn_token_kernel<T, RT, 1><<<ctas, kTileThreads, 0, s>>>(p);
    else if (w <= 64)
        xattn_token_kernel<T, RT, 2><<<ctas, kTileThreads, 0, s>>>(p);
    else
        xattn_token_kernel<T, RT, 4><<<ctas, kTileThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <class T>
cudaError_t fwd_rows(const AttnParams &p, cudaStream_t s) {
    if (p.unit_rows == 1) return token<T, 1>(p, s);
    if (p.unit_rows == 2) return token<T, 2>(p, s);
    if (p.unit_rows == 4) return token<T, 4>(p, s);
    return p.unit_rows == 16 ? fwd_width<T, 1>(p, s) : fwd_width<T, 4>(p, s);
}

template <class T, int U, int C>
cudaError_t grad(const AttnParams &p, cudaStream_t s) {
    constexpr int kept = 16 * U;
    const int w = tile_stride<C>(p.d) + tile_stride<C>(p.dv);
    const int key_blocks = (p.m + kept - 1) / kept, row_blocks = (p.n * p.group + kept - 1) / kept;
    const size_t fixed = (size_t)kept * w + 2 * kept * (kStream + 4) + 2 * kept;
    const size_t tile = (size_t)kStream * w + 2 * kStream;
    const int bufs = (fixed + 2 * tile) * sizeof(float) <= kMaxSmem ? 2 : 1;
    const size_t smem = (fixed + bufs * tile) * sizeof(float);
    cudaError_t e = allow_smem<&xattn_grad_kernel<T, U, C>>(smem);
    if (e != cudaSuccess) return e;
    const bool vec = aligned4<T>(p.q, p.qs) && aligned4<T>(p.k, p.ks) && aligned4<T>(p.v, p.vs) &&
                     aligned4<T>(p.dout, p.dos);
    xattn_grad_kernel<T, U, C>
        <<<dim3(key_blocks * p.key_parts + row_blocks * p.row_parts, p.batch * p.kv_heads), kTileThreads, smem, s>>>(
            p, vec, bufs, key_blocks);
    return cudaGetLastError();
}
template <class T, int U>
cudaError_t grad_width(const AttnParams &p, cudaStream_t s) {
    const int w = p.d > p.dv ? p.d : p.dv;
    return w <= 64 ? grad<T, U, 1>(p, s) : w <= 128 ? grad<T, U, 2>(p, s) : grad<T, U, 4>(p, s);
}
template <class T>
cudaError_t grad_rows(const AttnParams &p, int sms, cudaStream_t s) {
    return xattn_simt_rows(p.m + p.n * p.group, p.batch * p.kv_heads, sms) == 16 ? grad_width<T, 1>(p, s)
                                                                               : grad_width<T, 4>(p, s);
}

}  // namespace

bool xattn_token_ok(const void *q, const fs_view &qs, const void *k, const fs_view &ks, const void *v,
                    const fs_view &vs, int d, int dv, int rows, bool bf16) {
    if (rows > 8 || d > 128 || dv > 128 || d % 4 || dv % 4) return false;
    return bf16 ? aligned4<__nv_bfloat16>(q, qs) && aligned4<__nv_bfloat16>(k, ks) && aligned4<__nv_bfloat16>(v, vs)
                : aligned4<float>(q, qs) && aligned4<float>(k, ks) && aligned4<float>(v, vs);
}

cudaError_t launch_xattn_simt(const AttnParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? fwd_rows<__nv_bfloat16>(p, s) : fwd_rows<float>(p, s);
}
cudaError_t launch_xattn_combine(const AttnParams &p, bool bf16, cudaStream_t s) {
    const size_t rows = (size_t)p.tail_units * p.unit_rows;
    const unsigned grid = (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32));
    return bf16 ? launch_dependent(xattn_combine_kernel<__nv_bfloat16>, grid, kThreads, 0, s, p)
                : launch_dependent(xattn_combine_kernel<float>, grid, kThreads, 0, s, p);
}
cudaError_t launch_xattn_dot(const AttnParams &p, bool bf16, cudaStream_t s) {
    int per = 1;
    while (per < 32 && 8 * per < p.dv) per *= 2;
    const unsigned long long threads = (unsigned long long)p.n * p.heads * per;  // below 2^32: n heads < 2^27
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), p.batch);
    const bool vec = bf16 ? aligned4<__nv_bfloat16>(p.out, p.os) && aligned4<__nv_bfloat16>(p.dout, p.dos)
                          : aligned4<float>(p.out, p.os) && aligned4<float>(p.dout, p.dos);
    const auto kernel = bf16 ? xattn_dot_kernel<__nv_bfloat16> : xattn_dot_kernel<float>;
    // behind the statistics, which the row products do not need
    if (p.top) return launch_dependent(kernel, grid, kThreads, 0, s, p, per, vec);
    kernel<<<grid, kThreads, 0, s>>>(p, per, vec);
    return cudaGetLastError();
}
cudaError_t launch_xattn_grad_simt(const AttnParams &p, bool bf16, int sms, cudaStream_t s) {
    return bf16 ? grad_rows<__nv_bfloat16>(p, sms, s) : grad_rows<float>(p, sms, s);
}
cudaError_t launch_xattn_grad_join_simt(const AttnParams &p, bool bf16, cudaStream_t s) {
    const int rows = p.n * p.group, key_padded = (p.m + 15) / 16 * 16, row_padded = (rows + 15) / 16 * 16;
    const size_t work = (p.key_parts > 1 ? (size_t)p.m * (p.d + p.dv) : 0) + (p.row_parts > 1 ? (size_t)rows * p.d : 0);
    const dim3 grid((unsigned)((work + 255) / 256), p.batch * p.kv_heads);
    return bf16 ? launch_dependent(xattn_grad_join_simt_kernel<__nv_bfloat16>, grid, 256, 0, s, p, key_padded, row_padded)
                : launch_dependent(xattn_grad_join_simt_kernel<float>, grid, 256, 0, s, p, key_padded, row_padded);
}

}  // namespace fs
