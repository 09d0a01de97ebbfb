// Softmax cross entropy over a large vocabulary: what goes around the products
// of fs_xent_tc.cu -- operands that those cannot read as they lie, joining the
// partial statistics of a row, rounding dx.
//
//   z_ij = scale x_i.w_j,  lse_i = log sum_j e^{z_ij},  loss_i = lse_i - z_{i,t_i}
//   dz_ij = e^{z_ij - lse_i} (dloss_i + dlse_i) - [j = t_i] dloss_i
//   dx_i = scale sum_j dz_ij w_j,  dw_j = scale sum_i dz_ij x_i
//
// fp32 operands become three bf16 planes (each the rounding of what the ones
// before left, 8 significant bits a plane, 24 together) side by side in a row;
// the products then sum the six plane pairs that matter, (h h), (h m), (m h),
// (h l), (l h), (m m), and drop terms of 2^-24 of the whole.  bf16 operands
// whose rows a TMA box cannot start on are copied to an aligned plane.
#include "fs_ops.cuh"

namespace fs {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float *o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

// rows x d (row stride ld) -> rows x (PLANES dp) bf16, zeros beyond d; eight elements a thread.
template <class T, int PLANES>
__global__ void __launch_bounds__(256) xent_pack_kernel(const T *src, long long ld, int rows, int d, int dp, bool vec,
                                                        __nv_bfloat16 *dst) {
    const int per = dp / 8;
    for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < (size_t)rows * per; e += (size_t)gridDim.x * 256) {
        const size_t row = e / per;
        const int k = (int)(e % per) * 8;
        const T *p = src + (long long)row * ld + k;
        float v[8];
        if (sizeof(T) == 4 && vec && k + 8 <= d) {
            const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = k + u < d ? to_f(p[u]) : 0.f;
        }
#pragma unroll
        for (int pl = 0; pl < PLANES; ++pl) {
            __nv_bfloat16 h[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                h[u] = __float2bfloat16_rn(v[u]);
                v[u] -= __bfloat162float(h[u]);
            }
            *reinterpret_cast<uint4 *>(dst + (row * PLANES + pl) * dp + k) = *reinterpret_cast<const uint4 *>(h);
        }
    }
}

// The online states (max, sum) of two disjoint parts of a row, joined.
__device__ __forceinline__ void join(float &mx, float &l, float m2, float l2) {
    const float mn = fmaxf(mx, m2), ref = mn == -INFINITY ? 0.f : mn;
    l = l * exp2f(mx - ref) + l2 * exp2f(m2 - ref);
    mx = mn;
}

// Joins the column tiles of a row and writes lse and loss.  `per` threads of a
// warp take a row (a power of two), or the whole block takes one (per = 256):
// few rows have many tiles each and nothing else to run beside them.  The order
// of the sum depends on the sizes alone.
__global__ void __launch_bounds__(256) xent_finish_kernel(const XentParams p, int tiles, int per) {
    const long long g = (long long)blockIdx.x * 256 + threadIdx.x;
    const int sub = (int)(g % per);
    const long long i = g / per;
    const bool live = i < p.n;
    grid_dependency_wait();
    float mx = -INFINITY, l = 0.f;
    for (int t0 = sub; live && t0 < tiles; t0 += 4 * per) {
        float2 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = t0 + u * per < tiles ? p.part[(size_t)(t0 + u * per) * p.n + i] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int u = 0; u < 4; ++u) join(mx, l, v[u].x, v[u].y);
    }
    for (int s = min(per, 32) / 2; s; s >>= 1) {
        const float m2 = __shfl_down_sync(~0u, mx, s, 32), l2 = __shfl_down_sync(~0u, l, s, 32);
        join(mx, l, m2, l2);
    }
    if (per == 256) {
        __shared__ float2 warps[8];
        if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = make_float2(mx, l);
        __syncthreads();
        if (sub == 0)
            for (int w = 1; w < 8; ++w) join(mx, l, warps[w].x, warps[w].y);
    }
    if (!live || sub) return;
    const double lse = ((double)mx + log2((double)l)) * kLn2d;  // no sum at all: every logit was -inf, and so is lse
    p.lse[i] = (float)lse;
    const long long t = p.target[i];
    p.loss[i] = t == p.ignore ? 0.f : (t < 0 || t >= p.v ? NAN : (float)(lse - (double)p.hit[i]));
}

template <class T>
__global__ void __launch_bounds__(256) xent_reduce_kernel(const XentParams p) {
    const size_t all = (size_t)p.n * p.d;
    const float mul = p.scale_m * xent_unit(p);
    for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < all; e += (size_t)gridDim.x * 256) {
        float s = 0.f;
        const size_t i = e / p.d, j = e % p.d;
        for (int k = 0; k < p.parts; ++k) s += p.acc[((size_t)k * p.n + i) * p.ld_acc + j];
        from_f(s * mul, (T *)p.dx + p.lddx * (long long)i + (long long)j);
    }
}

}  // namespace

cudaError_t launch_xent_pack(const void *src, long long ld, int rows, int d, int dp, bool bf16, void *dst,
                             cudaStream_t s) {
    const size_t blocks = ((size_t)rows * (dp / 8) + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 8192 ? blocks : 8192);
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0 && ld % 4 == 0;
    if (bf16)
        xent_pack_kernel<__nv_bfloat16, 1>
            <<<grid, 256, 0, s>>>((const __nv_bfloat16 *)src, ld, rows, d, dp, false, (__nv_bfloat16 *)dst);
    else
        xent_pack_kernel<float, 3><<<grid, 256, 0, s>>>((const float *)src, ld, rows, d, dp, vec, (__nv_bfloat16 *)dst);
    return cudaGetLastError();
}
cudaError_t launch_xent_finish(const XentParams &p, int tiles, cudaStream_t s) {
    int per = 256;
    if (p.n > 512)
        for (per = 32; per > 1 && (long long)p.n * per > 1 << 16;) per /= 2;
    const long long threads = (long long)p.n * per;
    return launch_dependent(xent_finish_kernel, dim3((unsigned)((threads + 255) / 256)), 256, 0, s, p, tiles, per);
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
