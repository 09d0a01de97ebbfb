// Softmax cross entropy over a large vocabulary on CUDA cores, and the passes
// that both paths share (joining the partial statistics, rounding dx).
//
//   z_ij = scale x_i.w_j,  lse_i = log sum_j e^{z_ij},  loss_i = lse_i - z_{i,t_i}
//   dz_ij = e^{z_ij - lse_i} (dloss_i + dlse_i) - [j = t_i] dloss_i
//   dx_i = scale sum_j dz_ij w_j,  dw_j = scale sum_i dz_ij x_i
//
// One product kernel with three epilogues: C_ij = sum_k A_ik B_jk over 128 x
// 128 tiles, any element strides.  fp32 inputs always come here, and bf16
// inputs whose rows a TMA box cannot start on.
#include "fs_ops.cuh"

namespace fs {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float *o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

constexpr int kT = 128, kK = 16, kThreads = 256;
enum { kLse = 0, kDl = 1, kAcc = 2, kOut = 3 };

// C tile = A (rows i of `ni`, element strides sai, sak) B^T (rows j of `nj`), k in [k0, k1).
template <class TA, class TB, class TO, int EPI>
__global__ void __launch_bounds__(kThreads)
    product_kernel(const XentParams p, const TA *A, long long sai, long long sak, int ni, const TB *B, long long sbj,
                   long long sbk, int nj, int nk, int k_part, TO *out, long long ldo, float factor) {
    __shared__ __align__(16) float sA[kK][kT + 4], sB[kK][kT + 4];
    const int i0 = blockIdx.x * kT, j0 = blockIdx.y * kT;
    const int k0 = blockIdx.z * k_part, k1 = min(nk, k0 + k_part);
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float c[8][8];
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
        for (int b = 0; b < 8; ++b) c[a][b] = 0.f;
    for (int k = k0; k < k1; k += kK) {
        // consecutive threads run along whichever axis is contiguous
        for (int e = threadIdx.x; e < kT * kK; e += kThreads) {
            const int kk = sak == 1 ? e % kK : e / kT, r = sak == 1 ? e / kK : e % kT;
            sA[kk][r] = i0 + r < ni && k + kk < k1 ? to_f(A[sai * (i0 + r) + sak * (k + kk)]) : 0.f;
        }
        for (int e = threadIdx.x; e < kT * kK; e += kThreads) {
            const int kk = sbk == 1 ? e % kK : e / kT, r = sbk == 1 ? e / kK : e % kT;
            sB[kk][r] = j0 + r < nj && k + kk < k1 ? to_f(B[sbj * (j0 + r) + sbk * (k + kk)]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
            float a[8], b[8];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                *reinterpret_cast<float4 *>(a + 4 * u) = *reinterpret_cast<const float4 *>(&sA[kk][ti * 4 + 64 * u]);
                *reinterpret_cast<float4 *>(b + 4 * u) = *reinterpret_cast<const float4 *>(&sB[kk][tj * 4 + 64 * u]);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int w = 0; w < 8; ++w) c[u][w] = fmaf(a[u], b[w], c[u][w]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int i = i0 + ti * 4 + (u / 4) * 64 + u % 4;
        const bool live = i < ni;
        if constexpr (EPI == kLse) {
            const long long t = live ? p.target[i] : -1;
            float mx = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const int j = j0 + tj * 4 + (w / 4) * 64 + w % 4;
                if (live && j < nj && j == t) p.hit[i] = c[u][w] * p.scale;
                c[u][w] = j < nj ? c[u][w] * p.scale2 : -INFINITY;
                mx = fmaxf(mx, c[u][w]);
            }
            for (int s = 8; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, s));
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int w = 0; w < 8; ++w) l += exp2f(c[u][w] - ref);
            for (int s = 8; s; s >>= 1) l += __shfl_xor_sync(~0u, l, s);
            if (live && tj == 0) p.part[(size_t)blockIdx.y * ni + i] = make_float2(ref, l);
        } else if constexpr (EPI == kDl) {
            if (!live) continue;
            const long long t = p.target[i];
            const bool ign = t == p.ignore;
            const float gl = ign ? 0.f : (t < 0 || t >= p.v ? NAN : p.dloss[i]);
            const float gs = gl + (p.dlse ? p.dlse[i] : 0.f), l2 = p.lse[i] * kLog2e;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const int j = j0 + tj * 4 + (w / 4) * 64 + w % 4;
                if (j >= nj) continue;
                // a row without a gradient stays out even if its logits are not finite
                float g = gs == 0.f ? 0.f : exp2f(fmaf(c[u][w], p.scale2, -l2)) * gs;
                if (j + p.c0 == t && !ign) g -= gl;
                from_f(g * p.scale, out + ldo * i + j);
            }
        } else {
            if (!live) continue;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const int j = j0 + tj * 4 + (w / 4) * 64 + w % 4;
                if (j >= nj) continue;
                if constexpr (EPI == kAcc) {
                    float *o = p.acc + ((size_t)blockIdx.z * ni + i) * p.ld_acc + j;
                    *o = p.acc_add ? *o + c[u][w] : c[u][w];
                } else {
                    from_f(c[u][w] * factor, out + ldo * i + j);
                }
            }
        }
    }
}

// Joins the column tiles of a row in order and writes lse and loss.  `per`
// threads take a row (a power of two up to 32): one where there are many rows,
// a warp where there are few.
__global__ void __launch_bounds__(256) xent_finish_kernel(const XentParams p, int tiles, int per) {
    const long long g = (long long)blockIdx.x * 256 + threadIdx.x;
    const int sub = (int)(g % per);
    const long long i = g / per;
    const bool live = i < p.n;
    // the row's partial (max, sum) pairs: per neighbouring lanes take every per-th tile
    float mx = -INFINITY, l = 0.f;
    for (int t = sub; live && t < tiles; t += per) {
        const float2 v = p.part[(size_t)t * p.n + i];
        const float mn = fmaxf(mx, v.x);
        const float ref = mn == -INFINITY ? 0.f : mn;
        l = l * exp2f(mx - ref) + v.y * exp2f(v.x - ref);
        mx = mn;
    }
    for (int s = per / 2; s; s >>= 1) {
        const float m2 = __shfl_xor_sync(~0u, mx, s), l2 = __shfl_xor_sync(~0u, l, s);
        const float mn = fmaxf(mx, m2), ref = mn == -INFINITY ? 0.f : mn;
        const float la = l * exp2f(mx - ref), lb = l2 * exp2f(m2 - ref);
        l = (sub & s) ? lb + la : la + lb;  // the same order on both lanes
        mx = mn;
    }
    if (!live || sub) return;
    // no sum at all: every logit was NaN
    const double lse = l == 0.f ? (double)NAN : ((double)mx + log2((double)l)) * kLn2d;
    p.lse[i] = (float)lse;
    const long long t = p.target[i];
    p.loss[i] = t == p.ignore ? 0.f : (t < 0 || t >= p.v ? NAN : (float)(lse - (double)p.hit[i]));
}

template <class T>
__global__ void __launch_bounds__(256) xent_reduce_kernel(const XentParams p) {
    const size_t all = (size_t)p.n * p.d;
    for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < all; e += (size_t)gridDim.x * 256) {
        float s = 0.f;
        const size_t i = e / p.d, j = e % p.d;
        for (int k = 0; k < p.parts; ++k) s += p.acc[((size_t)k * p.n + i) * p.ld_acc + j];
        from_f(s, (T *)p.dx + p.lddx * (long long)i + (long long)j);
    }
}

int up(int a, int b) { return (a + b - 1) / b; }

template <class T>
cudaError_t lse(const XentParams &p, cudaStream_t s) {
    product_kernel<T, T, T, kLse><<<dim3(up(p.n, kT), up(p.v, kT)), kThreads, 0, s>>>(
        p, (const T *)p.x, p.ldx, 1, p.n, (const T *)p.w, p.ldw, 1, p.v, p.d, p.d, nullptr, 0, 1.f);
    return cudaGetLastError();
}
template <class T>
cudaError_t dl(const XentParams &p, cudaStream_t s) {
    const int nc = p.c1 - p.c0;
    product_kernel<T, T, float, kDl><<<dim3(up(p.n, kT), up(nc, kT)), kThreads, 0, s>>>(
        p, (const T *)p.x, p.ldx, 1, p.n, (const T *)p.w + p.ldw * p.c0, p.ldw, 1, nc, p.d, p.d, (float *)p.dl,
        p.ld_dl, 1.f);
    return cudaGetLastError();
}
template <class T>
cudaError_t dx(const XentParams &p, cudaStream_t s) {
    const int nc = p.c1 - p.c0;
    const int part = up(up(nc, p.parts), kK) * kK;
    product_kernel<float, T, float, kAcc><<<dim3(up(p.n, kT), up(p.d, kT), p.parts), kThreads, 0, s>>>(
        p, (const float *)p.dl, p.ld_dl, 1, p.n, (const T *)p.w + p.ldw * p.c0, 1, p.ldw, p.d, nc, part, nullptr, 0,
        1.f);
    return cudaGetLastError();
}
template <class T>
cudaError_t dw(const XentParams &p, cudaStream_t s) {
    const int nc = p.c1 - p.c0;
    product_kernel<float, T, T, kOut><<<dim3(up(nc, kT), up(p.d, kT)), kThreads, 0, s>>>(
        p, (const float *)p.dl, 1, p.ld_dl, nc, (const T *)p.x, 1, p.ldx, p.d, p.n, p.n, (T *)p.dw + p.lddw * p.c0,
        p.lddw, 1.f);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_xent_lse_simt(const XentParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? lse<__nv_bfloat16>(p, s) : lse<float>(p, s);
}
cudaError_t launch_xent_dl_simt(const XentParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? dl<__nv_bfloat16>(p, s) : dl<float>(p, s);
}
cudaError_t launch_xent_dx_simt(const XentParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? dx<__nv_bfloat16>(p, s) : dx<float>(p, s);
}
cudaError_t launch_xent_dw_simt(const XentParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? dw<__nv_bfloat16>(p, s) : dw<float>(p, s);
}
cudaError_t launch_xent_finish(const XentParams &p, int tiles, cudaStream_t s) {
    int per = 1;
    while (per < 32 && (long long)p.n * per < 1 << 15) per *= 2;
    const long long threads = (long long)p.n * per;
    xent_finish_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(p, tiles, per);
    return cudaGetLastError();
}
cudaError_t launch_xent_reduce(const XentParams &p, bool bf16, cudaStream_t s) {
    const size_t all = (size_t)p.n * p.d, blocks = (all + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 4096 ? blocks : 4096);
    if (bf16)
        xent_reduce_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    else
        xent_reduce_kernel<float><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace fs
