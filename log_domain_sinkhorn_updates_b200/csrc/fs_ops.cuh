// Internal declarations of the row-softmax operators beside the Sinkhorn
// passes: cross attention and softmax cross entropy, with their gradients.
#pragma once

#include <atomic>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "flashsinkhorn.h"
#include "fs_internal.cuh"

namespace fs {

// A bias at or below this masks its key (it counts as -inf).  Masks written as
// the type's lowest value then leave an empty row empty instead of making all
// of its keys equally likely, and times log2(e) no kept bias leaves fp32.
constexpr float kBiasMask = -1e30f;
// Biases are measured from the largest kept one where that is more than this in size (attn_top): against a bias of -1e9
// on every key of a problem (a sample masked with a finite constant), fp32 would lose the scores, and an LSE of that
// size the logarithm of the sum.  Up to it the largest costs the scores 2^-18 at most, and nothing is taken off.
constexpr float kBiasNear = 64.f;

// A row's statistics over one part of the keys: what the part's biases are measured from, the reference (base 2) of its
// scores beside them, and the sum.
struct alignas(16) AttnPart {
    float top, m, l;
};
constexpr int kAttnParts = 128;  // parts of a row at most

struct AttnParams {
    int batch, n, m, heads, kv_heads, group, d, dv;
    unsigned group_mul, group_shift;  // r / group without a division (row_query in fs_xattn.cu)
    float scale, scale2;  // score scale, and times log2(e)
    fs_view qs, ks, vs, os, dos, dqs, dks, dvs;  // element strides (batch, token, head)
    const void *q, *k, *v, *dout;
    const int *k_len;     // [batch] or null
    const float *bias;    // [batch][m] or null
    void *out, *dq, *dk, *dv_out;
    float *lse;           // [batch][heads][n], natural log (out of the forward, into the gradient); may be null forward
    float *dot;           // gradient: [batch][heads][n], D_i = dout_i.out_i
    float *lse2;          // gradient: [batch][heads][n], base-2 LSE measured from `top`
    float *top;           // gradient: [batch], what the problem's biases are measured from; null without a bias
    // 1: the forward's kernels, at a gradient's start, write top, and lse2 of the problems where it is large: there one
    // fp32 number does not hold the LSE, and the gradient cannot do with the forward's.  Their CTAs leave at once elsewhere.
    int stats;
    // Forward: a unit is unit_rows packed rows of a key head.  Units from main_units on are split over their keys into
    // `splits` parts of split_keys keys, a CTA each, which the joining pass adds up; 1: no unit is.
    int unit_rows, blocks;   // and the units of a head
    int main_units, tail_units, splits, split_keys;
    float *part_o;           // [splits][tail_units][unit_rows][dv], relative to part_ml's reference
    AttnPart *part_ml;       // [splits][tail_units][unit_rows]
    // Gradient: the streamed tiles of a CTA in parts, a CTA each (1: not split), whose raw sums
    // [part][batch kv_heads][padded rows][width] a joining pass adds up.
    int key_parts, row_parts;
    float *part_dk, *part_dv, *part_dq;
    unsigned long long timeout_ns;
    int *err;
};

// Allows a kernel `bytes` of dynamic shared memory, once a device (Kernel: one function, each with a list of its own).
// Sizes differ from call to call, so the limit only rises, under a lock: of two threads on first use the one that asks
// for less could otherwise set its limit last and the other record its own.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    static std::atomic<size_t> allowed[64];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && allowed[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && allowed[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) allowed[dev].store(bytes, std::memory_order_relaxed);
    return e;
}

// A kernel launched by launch_dependent may start before the stream's last one has ended (its launch then costs no
// gap); nothing that one wrote may be read before this wait.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... A, class... B>
cudaError_t launch_dependent(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, B... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Valid keys of problem b.
__device__ __forceinline__ int attn_keys(const AttnParams &p, int b) {
    return p.k_len ? min(max(__ldg(p.k_len + b), 0), p.m) : p.m;
}
// The problem of place `place` in the forward's order: with lengths, the longest first (ties: the lowest index), so
// that short ones fill in behind; as they come where there are more than 32.  By whole warps.  LENGTHS (p.k_len is
// given) is a template parameter where it matters: a problem that is not a function of the block index alone costs the
// tensor-core forward 4 %.
template <bool LENGTHS>
__device__ __forceinline__ int attn_problem(const AttnParams &p, int place) {
    if (!LENGTHS || p.batch > 32 || p.batch == 1) return place;
    const int lane = threadIdx.x & 31, len = lane < p.batch ? attn_keys(p, lane) : -1;
    int before = 0;
    for (int j = 0; j < p.batch; ++j) {
        const int other = __shfl_sync(~0u, len, j);
        before += other > len || (other == len && j < lane);
    }
    return __ffs(__ballot_sync(~0u, lane < p.batch && before == place)) - 1;
}

// The work of a CTA of the forward.
struct AttnUnit {
    int r0, c, b;       // first packed row, key head, problem
    int j_beg, j_end;   // its keys
    size_t part;        // first row of part_ml and part_o, where it is a part
    bool whole;
};
template <bool LENGTHS>
__device__ __forceinline__ AttnUnit attn_unit(const AttnParams &p) {
    AttnUnit w;
    const int x = blockIdx.x, t = x - p.main_units;
    w.whole = p.splits == 1 || t < 0;
    const int tu = w.whole ? 0 : t / p.splits, sp = w.whole ? 0 : t % p.splits;
    const int u = w.whole ? x : p.main_units + tu;
    w.r0 = u % p.blocks * p.unit_rows;
    w.c = u / p.blocks % p.kv_heads;
    w.b = attn_problem<LENGTHS>(p, u / p.blocks / p.kv_heads);
    const int keys = attn_keys(p, w.b);
    w.j_beg = sp * p.split_keys;
    w.j_end = w.whole ? keys : min(keys, w.j_beg + p.split_keys);
    w.part = ((size_t)sp * p.tail_units + tu) * p.unit_rows;
    return w;
}
// What the biases of keys [j_beg, j_end) of problem b are measured from: the largest kept one, or 0 where it is near 0;
// -inf where none is kept: the caller then takes no key at all, and a query of such a problem may hold anything.
// By a whole block of THREADS threads; scratch: a float a warp.
template <int THREADS>
__device__ __forceinline__ float attn_top(const AttnParams &p, int b, int j_beg, int j_end, float *scratch) {
    if (!p.bias) return 0.f;
    const float *bias = p.bias + (size_t)b * p.m;
    float top = -INFINITY;
#pragma unroll 8
    for (int j = j_beg + (int)threadIdx.x; j < j_end; j += THREADS) {
        const float v = __ldg(bias + j);
        if (v > kBiasMask) top = fmaxf(top, v);
    }
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = top;
    __syncthreads();
    for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, scratch[w]);
    __syncthreads();
    return fabsf(top) > kBiasNear ? top : 0.f;
}
// Statistics for a gradient (AttnParams::stats): whether the problem needs none.
__device__ __forceinline__ bool attn_stats_done(const AttnParams &p, const AttnUnit &unit, float top) {
    if (!p.stats) return false;
    if (threadIdx.x == 0 && unit.r0 == 0 && unit.c == 0) p.top[unit.b] = top;
    return top == 0.f || top == -INFINITY;
}
// Gradient: the keys of problem b that take part, as attn_top found them.
__device__ __forceinline__ int attn_grad_keys(const AttnParams &p, int b) {
    return p.top && p.top[b] == -INFINITY ? 0 : attn_keys(p, b);
}
// Base-2 bias of key j (valid or not), measured from top: -inf where it is masked.
__device__ __forceinline__ float attn_bias2(const AttnParams &p, int b, int j, int keys, float top) {
    if (j >= keys) return -INFINITY;
    if (!p.bias) return 0.f;
    const float v = __ldg(p.bias + (size_t)b * p.m + j);
    return v <= kBiasMask ? -INFINITY : (v - top) * kLog2e;
}
__device__ __forceinline__ bool attn_masked(const AttnParams &p, int b, int j, int keys) {
    return j >= keys || (p.bias && __ldg(p.bias + (size_t)b * p.m + j) <= kBiasMask);
}

// TMA map of a bf16 tensor of `dims` axes (innermost first, contiguous), 128-byte swizzle; strides in elements
// of the axes but the first.  False if the driver refuses it.
bool encode_bf16_map(CUtensorMap *map, const void *base, int dims, const long long *size, const long long *stride,
                     const int *box);

// Rows of a CTA of the CUDA-core kernels: 64, or 16 where 64 would leave SMs without a CTA.
inline int xattn_simt_rows(int rows, int heads, int sms) {
    return rows <= 16 || (long long)((rows + 63) / 64) * heads < sms ? 16 : 64;
}

// Geometry of the tensor-core attention kernels.
struct AttnTc {
    int datoms, vatoms;  // 64-element columns of d and dv
    int dv_pad;          // dv rounded up to 16
    int slots;           // ring of K and V tiles
    int k_head, k_batch, v_head, v_batch;  // 0: that axis of the map has one element
};
struct AttnGradTc {
    int d_pad, dv_pad;  // rounded up to 16
    int slots;          // ring of streamed tiles
    int key_blocks, row_blocks;  // units of the pass that keeps keys, and of the one that keeps rows (CTAs behind it)
    int q_head, q_batch, g_head, g_batch, k_head, k_batch, v_head, v_batch;  // as above (g: dout)
};
bool attn_tc_view(const void *base, const fs_view &s, int tokens, int heads, int batch, bool map);
bool attn_map(CUtensorMap *map, const void *base, const fs_view &s, int w, int tokens, int heads, int batch,
              int box_rows, int *hm, int *bm);
cudaError_t launch_xattn_tc(const AttnParams &p, cudaStream_t s);

cudaError_t launch_xattn_grad_tc(const AttnParams &p, cudaStream_t s);
cudaError_t launch_xattn_grad_join(const AttnParams &p, cudaStream_t s);  // where key_parts or row_parts > 1

cudaError_t launch_xattn_simt(const AttnParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_xattn_grad_join_simt(const AttnParams &p, bool bf16, cudaStream_t s);  // as launch_xattn_grad_join
// Whether the CUDA-core forward takes the few rows of a key head by the token kernel (units of 1, 2 or 4 rows).
bool xattn_token_ok(const void *q, const fs_view &qs, const void *k, const fs_view &ks, const void *v,
                    const fs_view &vs, int d, int dv, int rows, bool bf16);
cudaError_t launch_xattn_combine(const AttnParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_xattn_dot(const AttnParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_xattn_grad_simt(const AttnParams &p, bool bf16, int sms, cudaStream_t s);

// Softmax cross entropy: rows x [n][d] against classes w [v][d].
struct XentParams {
    int n, v, d;
    int n_all;                     // rows of the call (n: of the product)
    float scale, scale2;           // logit scale, and times log2(e)
    float scale_pow, scale_m;      // scale = scale_pow scale_m: a power of two, and 1 <= scale_m < 2
    // The operands as the products read them: bf16 rows of `planes` planes (1 for bf16, 3 for fp32), plane_x and
    // plane_w elements apart.
    const void *x, *w;             // w: of the classes from c0 on
    long long ldx, ldw;            // row strides in elements
    int planes, plane_x, plane_w;
    const long long *target;       // [n]
    long long ignore;
    float *loss, *lse;             // [n]
    const float *dloss, *dlse;     // [n] ([n] or null)
    void *dx, *dw;                 // dw: of the classes from c0 on
    long long lddx, lddw;
    // one product's launch
    int c0, c1;                    // classes of the piece
    float2 *part;                  // [column tiles][n]: (max, sum) in base 2
    float *hit;                    // [n] scaled logit of the target
    void *dl;                      // [n][planes][ld_dl] gradient of the logits of classes c0..c1, over scale_m xent_unit
    long long ld_dl;
    float *acc;                    // [parts][n][ld_acc] partial sums of dx
    long long ld_acc;
    int parts;                     // parts of the class range (dx)
    int acc_add;                   // 1: add to acc, 0: overwrite
    unsigned long long timeout_ns;
    int *err;
};

// A factor 1 <= u < 2 that stays out of the logit gradients, with scale_m, until the products' sums: the significand of
// dloss of the first counted row that has any.  Of a mean's gradient dloss is the same everywhere, and bf16 would round
// dloss (1 - p) of every target the same way, by up to 2^-8 of the whole gradient (2^-9 in the mean); without it a target
// gives p - 1, and the roundings are even in sign (8192 rows, 131072 classes of 2048: 0.0030 -> 0.0018 beside 64 bits).
// Only exponents stay in dz, so no range is lost.  By whole warps; rows past the first 16384 are not looked at.
__device__ __forceinline__ float xent_unit(const XentParams &p) {
    const int lane = threadIdx.x & 31, rows = min(p.n_all, 16384);
    for (int i0 = 0; i0 < rows; i0 += 256) {
        float g[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + 32 * u + lane;
            g[u] = i < rows && p.target[i] != p.ignore ? fabsf(p.dloss[i]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const unsigned has = __ballot_sync(~0u, g[u] > 0.f && g[u] < INFINITY);
            if (has)
                return __uint_as_float((__float_as_uint(__shfl_sync(~0u, g[u], __ffs(has) - 1)) & 0x7fffffu) | 0x3f800000u);
        }
    }
    return 1.f;
}

// Columns of the products' tiles, one partial statistic of a row each.
constexpr int kXentCols = 256;
// fp32: terms of a gradient's sum that one accumulator takes.  The tensor core truncates at each of its steps (16
// terms), so a long sum drifts towards zero; sums of sums are added with rounding.  Relative error of the fp32
// gradients at 1024 rows, 16384 classes: 5.1e-6 in one sum.
constexpr int kXentF32Terms = 2048;

// One product C [M][N] of the tensor-core kernel.
struct XentGemm {
    int M, N, K, mt, nt;     // sizes, and 256-row and 256-column tiles
    int parts, k_part;       // parts of K, and the length of one
    int segments;            // plane pairs summed (1, or 6 of the three planes)
    int a_plane, b_plane;    // elements from plane to plane of the operands
    int pairs;               // CTA pairs of the grid
    int a_rows;              // rows of a box of A (K contiguous)
    int vec;                 // out's rows can be written 16 bytes (1) or 32 (2) at a time
    int add;                 // fp32 out: 1: onto what it holds
    void *out;
    long long ldo;
};

// Copies rows into aligned bf16 planes of dp elements (1 of bf16, 3 of fp32).
cudaError_t launch_xent_pack(const void *src, long long ld, int rows, int d, int dp, bool bf16, void *dst,
                             cudaStream_t s);
bool xent_tc_rows(const void *p, long long ld, int rows);  // readable as they lie (bf16)
cudaError_t xent_tc_pairs(int *pairs);
cudaError_t launch_xent_lse(const XentParams &p, int pairs, cudaStream_t s);
cudaError_t launch_xent_finish(const XentParams &p, int tiles, cudaStream_t s);
cudaError_t launch_xent_dl(const XentParams &p, int pairs, cudaStream_t s);
cudaError_t launch_xent_dx(const XentParams &p, bool direct, int pairs, cudaStream_t s);
cudaError_t launch_xent_dw(const XentParams &whole, int r0, int r1, bool add, int pairs, cudaStream_t s);
// dx = sum over the parts of acc, rounded to the output type.
cudaError_t launch_xent_reduce(const XentParams &p, bool bf16, cudaStream_t s);

}  // namespace fs
