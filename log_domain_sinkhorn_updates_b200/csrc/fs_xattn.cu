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
// The heads that share a key head are rows of one problem: row r = i group + h.
// Keys past the length or masked by the bias are staged as zeros, so nothing
// that stands in their memory reaches a sum.
#include "fs_ops.cuh"

namespace fs {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 16, kKeys = 64;  // forward tile
constexpr int kGT = 32;                // gradient tile (rows and keys)
constexpr int kMaxD = 256;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float *o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

// Element offset of packed row r (of key head c, problem b) in a query-side tensor.
__device__ __forceinline__ long long row_off(const fs_view &s, const AttnParams &p, int b, int c, int r) {
    return s.batch * b + s.token * (r / p.group) + s.head * (c * p.group + r % p.group);
}
__device__ __forceinline__ size_t row_stat(const AttnParams &p, int b, int c, int r) {
    return ((size_t)b * p.heads + c * p.group + r % p.group) * p.n + r / p.group;
}

// rows [r0, r0 + cnt) of a query-side tensor into sm[cnt][w + 1] (zeros beyond the last row)
template <class T>
__device__ void stage_rows(float *sm, const T *src, const fs_view &s, const AttnParams &p, int b, int c, int r0, int cnt,
                           int w) {
    const int rows = p.n * p.group;
    for (int e = threadIdx.x; e < cnt * w; e += blockDim.x) {
        const int r = e / w, k = e % w;
        sm[r * (w + 1) + k] = r0 + r < rows ? to_f(src[row_off(s, p, b, c, r0 + r) + k]) : 0.f;
    }
}
// keys [j0, j0 + cnt) of a key-side tensor (zeros where bias2 says the key is masked)
template <class T>
__device__ void stage_keys(float *sm, const T *src, const fs_view &s, int b, int c, int j0, int cnt, int w,
                           const float *bias2) {
    for (int e = threadIdx.x; e < cnt * w; e += blockDim.x) {
        const int j = e / w, k = e % w;
        sm[j * (w + 1) + k] =
            bias2[j] == -INFINITY ? 0.f : to_f(src[s.batch * b + s.token * (j0 + j) + s.head * c + k]);
    }
}

// One CTA: 16 packed rows of a key head over one part of the keys.
template <class T>
__global__ void __launch_bounds__(kThreads) xattn_simt_kernel(const AttnParams p) {
    extern __shared__ float sm[];
    const int tiles = (p.n * p.group + kRows - 1) / kRows;
    const int r0 = (blockIdx.x % tiles) * kRows, sp = blockIdx.x / tiles;
    const int c = blockIdx.y % p.kv_heads, b = blockIdx.y / p.kv_heads;
    float *sQ = sm, *sK = sQ + kRows * (p.d + 1), *sV = sK + kKeys * (p.d + 1);
    float *sP = sV + kKeys * (p.dv + 1), *sB = sP + kRows * (kKeys + 1);
    const int keys = attn_keys(p, b);
    const int j_beg = sp * p.split_keys, j_end = min(keys, j_beg + p.split_keys);
    stage_rows(sQ, (const T *)p.q, p.qs, p, b, c, r0, kRows, p.d);
    const int row = threadIdx.x / 8, t8 = threadIdx.x % 8;
    float o[kMaxD / 8];
#pragma unroll
    for (int k = 0; k < kMaxD / 8; ++k) o[k] = 0.f;
    float mx = -INFINITY, l = 0.f;
    for (int j0 = j_beg; j0 < j_end; j0 += kKeys) {
        __syncthreads();
        if (threadIdx.x < kKeys) sB[threadIdx.x] = attn_bias2(p, b, j0 + threadIdx.x, j_end);
        __syncthreads();
        stage_keys(sK, (const T *)p.k, p.ks, b, c, j0, kKeys, p.d, sB);
        stage_keys(sV, (const T *)p.v, p.vs, b, c, j0, kKeys, p.dv, sB);
        __syncthreads();
        float z[8], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] = 0.f;
        for (int k = 0; k < p.d; ++k) {
            const float qv = sQ[row * (p.d + 1) + k];
#pragma unroll
            for (int u = 0; u < 8; ++u) z[u] = fmaf(qv, sK[(t8 + 8 * u) * (p.d + 1) + k], z[u]);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            z[u] = fmaf(z[u], p.scale2, sB[t8 + 8 * u]);
            top = fmaxf(top, z[u]);
        }
        for (int w = 4; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
        const float mn = fmaxf(mx, top);
        const float ref = mn == -INFINITY ? 0.f : mn;  // nothing but masked keys so far: every term below is 0
        const float cor = exp2f(mx - ref);
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float e = exp2f(z[u] - ref);
            sP[row * (kKeys + 1) + t8 + 8 * u] = e;
            sum += e;
        }
        for (int w = 4; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        l = l * cor + sum;
        mx = mn;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kMaxD / 8; ++k) {
            const int e = t8 + 8 * k;
            if (e < p.dv) {
                float a = o[k] * cor;
                for (int j = 0; j < kKeys; ++j) a = fmaf(sP[row * (kKeys + 1) + j], sV[j * (p.dv + 1) + e], a);
                o[k] = a;
            }
        }
    }
    const int r = r0 + row;
    if (r >= p.n * p.group) return;
    if (p.splits > 1) {
        const size_t at = ((size_t)(sp * p.batch + b) * p.kv_heads + c) * p.n * p.group + r;
        if (t8 == 0) p.part_ml[at] = make_float2(mx, l);
        for (int k = 0; t8 + 8 * k < p.dv; ++k) p.part_o[at * p.dv + t8 + 8 * k] = o[k];
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: no key is left (a NaN row stays NaN)
    T *dst = (T *)p.out + row_off(p.os, p, b, c, r);
#pragma unroll
    for (int k = 0; k < kMaxD / 8; ++k)
        if (t8 + 8 * k < p.dv) from_f(o[k] * inv, dst + t8 + 8 * k);
    if (p.lse && t8 == 0)
        p.lse[row_stat(p, b, c, r)] = l == 0.f ? -INFINITY : (float)(((double)mx + log2((double)l)) * kLn2d);
}

// Joins the parts of a row, in the parts' order.  One warp per packed row.
template <class T>
__global__ void __launch_bounds__(kThreads) xattn_combine_kernel(const AttnParams p) {
    const size_t rows = (size_t)p.n * p.group, all = rows * p.batch * p.kv_heads;
    const size_t at = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (at >= all) return;
    const int lane = threadIdx.x % 32;
    const int r = (int)(at % rows), c = (int)(at / rows % p.kv_heads), b = (int)(at / rows / p.kv_heads);
    grid_dependency_wait();
    float mx = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) mx = fmaxf(mx, p.part_ml[s * all + at].x);
    for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float l = 0.f, o[kMaxD / 32];
#pragma unroll
    for (int k = 0; k < kMaxD / 32; ++k) o[k] = 0.f;
    for (int s0 = 0; s0 < p.splits; s0 += 32) {
        // a lane's part: its weight; 0 where it has no key (its sums were not written)
        const float2 ml = s0 + lane < p.splits ? p.part_ml[(s0 + lane) * all + at] : make_float2(-INFINITY, 0.f);
        const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - ref);
        const unsigned has = __ballot_sync(~0u, ml.y != 0.f);
        float lw = ml.y * f;
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
        p.lse[row_stat(p, b, c, r)] = l == 0.f ? -INFINITY : (float)(((double)mx + log2((double)l)) * kLn2d);
}

// D_i = dout_i.out_i, one warp per (problem, head, query).
template <class T>
__global__ void __launch_bounds__(kThreads) xattn_dot_kernel(const AttnParams p) {
    const size_t at = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (at >= (size_t)p.batch * p.n * p.heads) return;
    const int lane = threadIdx.x % 32;
    const int h = (int)(at % p.heads), i = (int)(at / p.heads % p.n), b = (int)(at / p.heads / p.n);
    const T *o = (const T *)p.out + p.os.batch * b + p.os.token * i + p.os.head * h;
    const T *g = (const T *)p.dout + p.dos.batch * b + p.dos.token * i + p.dos.head * h;
    float s = 0.f;
    for (int k = lane; k < p.dv; k += 32) s = fmaf(to_f(o[k]), to_f(g[k]), s);
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
    if (lane == 0) p.dot[((size_t)b * p.heads + h) * p.n + i] = s;
}

// The 32 x 32 tile of P and of dS: sP, sS [key][row] (rows past the end and masked keys: zero).
__device__ void grad_tile(const AttnParams &p, const float *sQ, const float *sG, const float *sK, const float *sV,
                          const float *sB, const float *sL, const float *sD, float *sP, float *sS) {
    for (int e = threadIdx.x; e < kGT * kGT; e += kThreads) {
        const int j = e / kGT, r = e % kGT;
        float s = 0.f, g = 0.f;
        for (int k = 0; k < p.d; ++k) s = fmaf(sQ[r * (p.d + 1) + k], sK[j * (p.d + 1) + k], s);
        for (int k = 0; k < p.dv; ++k) g = fmaf(sG[r * (p.dv + 1) + k], sV[j * (p.dv + 1) + k], g);
        const bool off = sB[j] == -INFINITY || sL[r] == INFINITY;
        const float pr = off ? 0.f : exp2f(fmaf(s, p.scale2, sB[j]) - sL[r]);
        sP[j * (kGT + 1) + r] = pr;
        sS[j * (kGT + 1) + r] = off ? 0.f : pr * (g - sD[r]);
    }
}
// Base-2 LSE and D of rows r0.. (an empty row, or one past the end, is marked by +inf).
__device__ void stage_stats(const AttnParams &p, int b, int c, int r0, float *sL, float *sD) {
    if (threadIdx.x < kGT) {
        const int r = r0 + threadIdx.x;
        float l = INFINITY, dd = 0.f;
        if (r < p.n * p.group) {
            const float v = p.lse[row_stat(p, b, c, r)];
            l = v == -INFINITY ? INFINITY : v * kLog2e;
            dd = p.dot[row_stat(p, b, c, r)];
        }
        sL[threadIdx.x] = l;
        sD[threadIdx.x] = dd;
    }
}

// KEYS: one CTA per 32 keys of a key head, over all its rows: dk and dv.
// Otherwise: one CTA per 32 packed rows, over all keys: dq.
template <class T, bool KEYS>
__global__ void __launch_bounds__(kThreads) xattn_grad_kernel(const AttnParams p) {
    extern __shared__ float sm[];
    const int c = blockIdx.y % p.kv_heads, b = blockIdx.y / p.kv_heads, t0 = blockIdx.x * kGT;
    float *sQ = sm, *sG = sQ + kGT * (p.d + 1), *sK = sG + kGT * (p.dv + 1), *sV = sK + kGT * (p.d + 1);
    float *sP = sV + kGT * (p.dv + 1), *sS = sP + kGT * (kGT + 1), *sB = sS + kGT * (kGT + 1), *sL = sB + kGT,
          *sD = sL + kGT;
    const int keys = attn_keys(p, b), rows = p.n * p.group;
    const int end = KEYS ? rows : keys;
    const int own = threadIdx.x / 4, t4 = threadIdx.x % 4;
    float a1[kMaxD / 4], a2[KEYS ? kMaxD / 4 : 1];
#pragma unroll
    for (int k = 0; k < kMaxD / 4; ++k) a1[k] = 0.f;
    if (KEYS) {
#pragma unroll
        for (int k = 0; k < (KEYS ? kMaxD / 4 : 1); ++k) a2[k] = 0.f;
        if (threadIdx.x < kGT) sB[threadIdx.x] = attn_bias2(p, b, t0 + threadIdx.x, keys);
        __syncthreads();
        stage_keys(sK, (const T *)p.k, p.ks, b, c, t0, kGT, p.d, sB);
        stage_keys(sV, (const T *)p.v, p.vs, b, c, t0, kGT, p.dv, sB);
    } else {
        stage_rows(sQ, (const T *)p.q, p.qs, p, b, c, t0, kGT, p.d);
        stage_rows(sG, (const T *)p.dout, p.dos, p, b, c, t0, kGT, p.dv);
        stage_stats(p, b, c, t0, sL, sD);
    }
    for (int u0 = 0; u0 < end; u0 += kGT) {
        __syncthreads();
        if (KEYS) {
            stage_rows(sQ, (const T *)p.q, p.qs, p, b, c, u0, kGT, p.d);
            stage_rows(sG, (const T *)p.dout, p.dos, p, b, c, u0, kGT, p.dv);
            stage_stats(p, b, c, u0, sL, sD);
        } else {
            if (threadIdx.x < kGT) sB[threadIdx.x] = attn_bias2(p, b, u0 + threadIdx.x, keys);
            __syncthreads();
            stage_keys(sK, (const T *)p.k, p.ks, b, c, u0, kGT, p.d, sB);
            stage_keys(sV, (const T *)p.v, p.vs, b, c, u0, kGT, p.dv, sB);
        }
        __syncthreads();
        grad_tile(p, sQ, sG, sK, sV, sB, sL, sD, sP, sS);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMaxD / 4; ++k) {
            const int e = t4 + 4 * k;
            if (e < p.d) {
                float s = a1[k];
                for (int u = 0; u < kGT; ++u)
                    s = KEYS ? fmaf(sS[own * (kGT + 1) + u], sQ[u * (p.d + 1) + e], s)
                             : fmaf(sS[u * (kGT + 1) + own], sK[u * (p.d + 1) + e], s);
                a1[k] = s;
            }
            if (KEYS && e < p.dv) {
                float s = a2[KEYS ? k : 0];
                for (int u = 0; u < kGT; ++u) s = fmaf(sP[own * (kGT + 1) + u], sG[u * (p.dv + 1) + e], s);
                a2[KEYS ? k : 0] = s;
            }
        }
    }
    const int at = t0 + own;
    if (KEYS) {
        if (at >= p.m) return;  // keys past the length get zeros: they take no part
        T *dk = (T *)p.dk + p.dks.batch * b + p.dks.token * at + p.dks.head * c;
        T *dv = (T *)p.dv_out + p.dvs.batch * b + p.dvs.token * at + p.dvs.head * c;
#pragma unroll
        for (int k = 0; k < kMaxD / 4; ++k) {
            if (t4 + 4 * k < p.d) from_f(a1[k] * p.scale, dk + t4 + 4 * k);
            if (t4 + 4 * k < p.dv) from_f(a2[KEYS ? k : 0], dv + t4 + 4 * k);
        }
    } else {
        if (at >= rows) return;
        T *dq = (T *)p.dq + row_off(p.dqs, p, b, c, at);
#pragma unroll
        for (int k = 0; k < kMaxD / 4; ++k)
            if (t4 + 4 * k < p.d) from_f(a1[k] * p.scale, dq + t4 + 4 * k);
    }
}

template <class K>
cudaError_t with_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <class T>
cudaError_t fwd(const AttnParams &p, cudaStream_t s) {
    const size_t smem =
        sizeof(float) * ((size_t)(kRows + kKeys) * (p.d + 1) + kKeys * (p.dv + 1) + kRows * (kKeys + 1) + kKeys);
    cudaError_t e = with_smem(xattn_simt_kernel<T>, smem);
    if (e != cudaSuccess) return e;
    const int tiles = (p.n * p.group + kRows - 1) / kRows;
    xattn_simt_kernel<T><<<dim3(tiles * p.splits, p.batch * p.kv_heads), kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <class T>
cudaError_t grad(const AttnParams &p, cudaStream_t s) {
    const size_t smem = sizeof(float) * ((size_t)2 * kGT * (p.d + 1 + p.dv + 1) + 2 * kGT * (kGT + 1) + 3 * kGT);
    cudaError_t e = with_smem(xattn_grad_kernel<T, true>, smem);
    if (e == cudaSuccess) e = with_smem(xattn_grad_kernel<T, false>, smem);
    if (e != cudaSuccess) return e;
    if (p.m > 0)
        xattn_grad_kernel<T, true><<<dim3((p.m + kGT - 1) / kGT, p.batch * p.kv_heads), kThreads, smem, s>>>(p);
    if (p.n > 0)
        xattn_grad_kernel<T, false><<<dim3((p.n * p.group + kGT - 1) / kGT, p.batch * p.kv_heads), kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_xattn_simt(const AttnParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? fwd<__nv_bfloat16>(p, s) : fwd<float>(p, s);
}
cudaError_t launch_xattn_combine(const AttnParams &p, bool bf16, cudaStream_t s) {
    const size_t rows = (size_t)p.n * p.group * p.batch * p.kv_heads;
    const unsigned grid = (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32));
    return bf16 ? launch_dependent(xattn_combine_kernel<__nv_bfloat16>, grid, kThreads, 0, s, p)
                : launch_dependent(xattn_combine_kernel<float>, grid, kThreads, 0, s, p);
}
cudaError_t launch_xattn_dot(const AttnParams &p, bool bf16, cudaStream_t s) {
    const size_t rows = (size_t)p.batch * p.n * p.heads;
    const unsigned grid = (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32));
    if (bf16)
        xattn_dot_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else
        xattn_dot_kernel<float><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
cudaError_t launch_xattn_grad_simt(const AttnParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? grad<__nv_bfloat16>(p, s) : grad<float>(p, s);
}

}  // namespace fs
