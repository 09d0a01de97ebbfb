// Softmax cross entropy on the sm_100a tensor cores: the three products of the
// operator (logits, dx, dw) as one persistent kernel on CTA pairs with an
// epilogue each, so that logits live in TMEM only and what leaves a tile is
// two numbers a row (forward) or the bf16 logit gradients of one piece of the
// classes (gradient).
//
//   LSE  C = x w^T          rows: (max, sum 2^(z - max)) per 256 columns, the target's logit
//   DL   C = x w^T          dz = scale (e^{z - lse} (dloss + dlse) - onehot dloss) -> bf16,
//                           the type of x and w, with which it is multiplied next; a
//                           factor common to all rows stays out of it (xent_unit)
//   ACC  C = dz w           fp32 partial sums of dx (per part of the classes)
//   OUT  C = dz^T x or dz w  rows of dw, or of dx where one product is all of it
//
// fp32 operands arrive as three bf16 planes (fs_xent.cu); dz is then written
// as three planes too, and a product's K runs over six plane pairs.
//
// One tcgen05.mma.cta_group::2 covers a 256 x 256 tile of the pair (each CTA
// holds 128 rows of A and 128 rows of B, and its own 128 x 256 accumulator, two
// of them in TMEM's 512 columns): per 64 columns of K a CTA reads 32 KB for 512
// cycles of MMA, where a 128 x 256 tile of one CTA would read 48 KB.  dz^T and
// w as the right factor are read as they lie: an operand whose M or N axis is
// contiguous is staged as 64-element columns by the same 128-byte swizzle and
// told apart by the descriptor (no transposed copy of x, w or dz is made).
// Warp 0 loads, warp 1 issues, two groups of four warps take alternate tiles
// out of TMEM, so an epilogue has two tiles' time before the MMAs wait for it.
#include <cuda.h>

#include "fs_ops_tc.cuh"

namespace fs {
namespace {

using namespace tc;

constexpr int kTile = 256, kBK = 64, kStages = 6;
constexpr int kOperand = 128 * kBK * 2;      // bytes of a CTA's share of one operand of a stage
constexpr int kStageBytes = 2 * kOperand;
constexpr int kThreads = 320;
constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
constexpr int kGroupRows = 8;  // row tiles that share a column tile while it is in L2

enum { kLse = 0, kDl = 1, kAcc = 2, kOut = 3 };

// The planes of A and of B in plane pair s: (m m), (l h), (h l), (m h), (h m), (h h).  The accumulator truncates at
// each step of K, by its own size: the small pairs go first, while it is small, and the steps that count are those of
// the last pair alone.
__device__ __forceinline__ int plane_a(int s) { return 0x049 >> (2 * s) & 3; }
__device__ __forceinline__ int plane_b(int s) { return 0x121 >> (2 * s) & 3; }

__device__ __forceinline__ void st_v8(void *p, const uint32_t *r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void ld_v8(const void *p, uint32_t *r) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
}
struct Tile {
    int m0, n0, k0, kb, part;  // first row and column, first K element, K blocks of a plane pair, part
};
__device__ __forceinline__ Tile tile_of(const XentGemm &g, int t) {
    Tile o;
    if (g.mt == 1 && g.parts == 1) {  // one row tile: no divisions between the loads of two tiles
        o.part = o.m0 = o.k0 = 0;
        o.n0 = t * kTile;
        o.kb = (g.K + kBK - 1) / kBK;
        return o;
    }
    const int per_part = g.mt * g.nt;
    o.part = t / per_part;
    const int r = t % per_part;
    const int band = r / (kGroupRows * g.nt), rows = min(kGroupRows, g.mt - band * kGroupRows);
    const int in = r - band * kGroupRows * g.nt;
    o.m0 = (band * kGroupRows + in % rows) * kTile;
    o.n0 = in / rows * kTile;
    o.k0 = o.part * g.k_part;
    o.kb = max(0, (min(g.K - o.k0, g.k_part) + kBK - 1) / kBK);
    return o;
}

// 128 columns [c, c + 128) of a row from TMEM.
__device__ __forceinline__ void load128(uint32_t ta, uint32_t (&r)[128]) {
    tmem_ld32(ta + 0u, &r[0]);
    tmem_ld32(ta + 32u, &r[32]);
    tmem_ld32(ta + 64u, &r[64]);
    tmem_ld32(ta + 96u, &r[96]);
    tmem_ld_wait();
}

// F32: three planes in, fp32 out.
template <int EPI, bool A_MN, bool B_MN, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    xent_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const XentParams p, const XentGemm g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);  // used in the first CTA
    uint64_t *empty = full + kStages;                                             // both CTAs
    uint64_t *sfull = empty + kStages;                                            // [2] both CTAs
    uint64_t *sempty = sfull + 2;                                                 // [2] first CTA (8 arrivals)
    uint64_t *drain = sempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(drain + 2);

    const uint32_t rank = cluster_rank();
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles = g.mt * g.nt * g.parts;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sfull + b, 1);
            mbar_init(sempty + b, 8);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // Few rows: only those of A are loaded (a box of zeros costs more than rows that exist: 145 us against 128 for one
    // row and 256 at 262144 classes of 1024), over zeros that stay.
    const int a_rows = A_MN ? 128 : g.a_rows;
    if (!A_MN && a_rows < 128)
        for (int e = threadIdx.x; e < kStages * kOperand / 16; e += kThreads)
            *reinterpret_cast<uint4 *>(smem + e / (kOperand / 16) * kStageBytes + e % (kOperand / 16) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
    fence_async();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_holder)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int i = 0;  // stages filled so far
            RingPos rp{0, 0};
            for (int t = pair; ok && t < tiles; t += pairs) {
                const Tile T = tile_of(g, t);
                const int ra = T.m0 + (int)rank * 128, rb = T.n0 + (int)rank * 128;
                const bool second = a_rows == 128;  // the second CTA has rows to load
                if (*abort_flag) break;
                int seg = 0, kb = -1;
                for (int u = 0; u < T.kb * g.segments; ++u, ++i) {
                    if (++kb == T.kb) {
                        kb = 0;
                        ++seg;
                    }
                    const int s = rp.slot, k = T.k0 + kb * kBK;
                    const int xa = F32 ? plane_a(seg) * g.a_plane : 0, xb = F32 ? plane_b(seg) * g.b_plane : 0;
                    if (i >= kStages && !mbar_wait_near(empty + s, rp.phase ^ 1u, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0)
                        mbar_expect_tx(full + s, 2u * kOperand + (second ? 2u * kOperand : (uint32_t)a_rows * 128u));
                    const uint32_t bar = cluster_addr(saddr(full + s), 0);
                    const uint32_t a = saddr(smem + s * kStageBytes), b = a + kOperand;
                    if (A_MN) {
                        tma_load_2d_pair(a, &map_a, bar, xa + ra, k);
                        tma_load_2d_pair(a + 8192u, &map_a, bar, xa + ra + 64, k);
                    } else if (rank == 0 || second) {
                        tma_load_2d_pair(a, &map_a, bar, xa + k, ra);
                    }
                    if (B_MN) {
                        tma_load_2d_pair(b, &map_b, bar, xb + rb, k);
                        tma_load_2d_pair(b + 8192u, &map_b, bar, xb + rb + 64, k);
                    } else {
                        tma_load_2d_pair(b, &map_b, bar, xb + k, rb);
                    }
                    rp.step(1, kStages);
                }
            }
            if (!ok) {
                atomicOr(p.err, kDevErrTimeout);
                *abort_flag = 1;
            }
            // never leave with copies in flight: both CTAs' copies count on the first one's barriers
            if (rank == 0)
                for (int j = max(0, i - kStages); j < i; ++j)
                    mbar_wait_near(full + (j % kStages), (uint32_t)(j / kStages) & 1u, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {  // the warp stays converged: elect_lane
            const bool lead = elect_lane();
            const uint32_t idesc = make_idesc<0, 256, 256>() | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
            constexpr uint32_t ka = A_MN ? 128u : 2u, kb16 = B_MN ? 128u : 2u;  // 16 of K, in 16-byte units
            const uint32_t base = saddr(smem);
            const uint64_t a0 = A_MN ? sdesc_mn(base, 8192u) : make_sdesc(base, 128u);
            const uint64_t b0 = B_MN ? sdesc_mn(base + kOperand, 8192u) : make_sdesc(base + kOperand, 128u);
            bool ok = true;
            RingPos rp{0, 0};
            int n = 0;
            for (int t = pair; ok && t < tiles; t += pairs, ++n) {
                const int blocks = tile_of(g, t).kb * g.segments;
                const int b = n & 1;
                if (n >= 2 && !warp_all(mbar_wait_cluster(sempty + b, ((uint32_t)(n >> 1) & 1u) ^ 1u, p.timeout_ns)))
                    ok = false;
                const uint32_t dt = tmem_base + (uint32_t)(b * 256);
                for (int kb = 0; ok && kb < blocks; ++kb) {
                    const bool aborted = *abort_flag;  // read under the wait
                    if (!warp_all(mbar_wait_near(full + rp.slot, rp.phase, p.timeout_ns) && !aborted)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (lead) {
                        const uint64_t ad = a0 + (uint64_t)(rp.slot * (kStageBytes >> 4));
                        const uint64_t bd = b0 + (uint64_t)(rp.slot * (kStageBytes >> 4));
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)
                            tc_mma_pair<0>(dt, ad + (uint64_t)(k * ka), bd + (uint64_t)(k * kb16), idesc,
                                           kb > 0 || k > 0 ? 1u : 0u);
                        tc_commit_pair(saddr(empty + rp.slot), (uint16_t)3);
                        if (kb == blocks - 1) tc_commit_pair(saddr(sfull + b), (uint16_t)3);
                    }
                    __syncwarp();
                    rp.step(1, kStages);
                }
                if (ok && blocks == 0 && lead) tc_commit_pair(saddr(sfull + b), (uint16_t)3);
            }
            if (lead) {
                if (!ok) {
                    atomicOr(p.err, kDevErrTimeout);
                    *abort_flag = 1;
                }
                tc_commit_pair(saddr(drain), (uint16_t)1);
            }
            __syncwarp();
            mbar_wait_near(drain, 0, p.timeout_ns);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, grp = (warp - 2) >> 2;
        const int rl = (int)rank * 128 + q * 32 + lane;
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(grp * 256);
        const uint32_t sempty0 = cluster_addr(saddr(sempty + grp), 0);
        const float unit = EPI == kDl || EPI == kOut ? xent_unit(p) : 1.f, mul = p.scale_m * unit;
        bool ok = true;
        int n = grp;
        for (int t = pair + grp * pairs; t < tiles; t += 2 * pairs, n += 2) {
            const Tile T = tile_of(g, t);
            const int row = T.m0 + rl;
            const bool live = row < g.M;
            // what the row needs, fetched while the MMAs run
            long long target = -1;
            float gl = 0.f, gs = 0.f, l2 = 0.f, l2lo = 0.f;
            if (EPI <= kDl && live) {
                target = __ldg(p.target + row);
                if (EPI == kDl) {
                    const bool ign = target == p.ignore;
                    gl = ign ? 0.f : (target < 0 || target >= p.v ? NAN : __ldg(p.dloss + row));
                    gs = (gl + (p.dlse ? __ldg(p.dlse + row) : 0.f)) / unit;
                    gl /= unit;  // exact where dloss is the common one
                    const float lse = __ldg(p.lse + row);
                    l2 = lse * kLog2e;
                    if (F32)  // what the product's rounding lost, and log2(e)'s own tail
                        l2lo = fmaf(lse, kLog2e, -l2) + lse * (float)(kLog2ed - (double)kLog2e);
                    if (ign) target = -1;
                }
            }
            const bool aborted = *abort_flag;  // read under the wait
            if (!warp_all(mbar_wait_near(sfull + grp, (uint32_t)(n >> 1) & 1u, p.timeout_ns) && !aborted)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float mx = -INFINITY, l = 0.f;
            if (T.m0 + (int)rank * 128 + q * 32 >= g.M) {  // none of the warp's rows exists
                if (lane == 0) mbar_arrive_cluster(sempty0);
                continue;
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int c0 = T.n0 + 128 * half;  // first column of the half
                uint32_t r[128];
                if (T.kb > 0) {
                    load128(taddr + 128u * half, r);
                } else {  // an empty sum: nothing was multiplied
#pragma unroll
                    for (int k = 0; k < 128; ++k) r[k] = 0u;
                }
                if (half == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(sempty0);
                }
                if (c0 >= g.N && !(EPI == kDl && F32)) continue;
                if constexpr (EPI == kLse) {
                    const long long at = target - p.c0 - c0;
                    if (__any_sync(~0u, at >= 0 && at < 128)) {
                        float hit = 0.f;
#pragma unroll
                        for (int k = 0; k < 128; ++k)
                            if (k == at) hit = __uint_as_float(r[k]);
                        if (at >= 0 && at < 128) p.hit[row] = hit * p.scale;
                    }
                    if (c0 + 128 > g.N) {
#pragma unroll
                        for (int k = 0; k < 128; ++k)
                            if (c0 + k >= g.N) r[k] = 0xff800000u;  // -inf
                    }
                    if (half == 0) {
                        // a first reference from 16 columns: where they are typical, the tile needs no pass for its
                        // maximum (a sum past 2^12 against it brings one)
                        float a = max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]));
                        float b = max3(__uint_as_float(r[3]), __uint_as_float(r[4]), __uint_as_float(r[5]));
#pragma unroll
                        for (int k = 6; k < 16; k += 4) {
                            a = max3(a, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                            if (k + 3 < 16) b = max3(b, __uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
                        }
                        mx = fmaxf(a, b) * p.scale2;
                        if (!(fabsf(mx) < INFINITY)) mx = -INFINITY;
                    }
                    consume128_folded(r, p.scale2, mx, l);
                } else if constexpr (EPI == kDl) {
                    const long long at = target - p.c0 - c0;
                    const bool any = __any_sync(~0u, at >= 0 && at < 128);
                    const int planes = F32 ? 3 : 1;
                    uint8_t *dst = (uint8_t *)p.dl + ((size_t)row * planes * p.ld_dl + c0) * 2;
#pragma unroll
                    for (int k = 0; k < 128; k += 16) {
                        float v[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            // a row without a gradient stays out even if its logits are not finite
                            float z = fmaf(__uint_as_float(r[k + u]), p.scale2, -l2);
                            if (F32) z -= l2lo;
                            v[u] = gs == 0.f ? 0.f : ex2_approx(z) * gs;
                            if (any && at == k + u) v[u] -= gl;
                            v[u] *= p.scale_pow;
                        }
                        // a row's padding beyond the last class (ld_dl is a multiple of 256) is written too: zeros
                        // where a next plane follows it, which the dx product reads
                        if (F32) {
                            if (c0 + 128 > g.N) {
#pragma unroll
                                for (int u = 0; u < 16; ++u)
                                    if (c0 + k + u >= g.N) v[u] = 0.f;
                            }
#pragma unroll
                            for (int pl = 0; pl < 3; ++pl) {
                                uint32_t w[8];
#pragma unroll
                                for (int u = 0; u < 16; u += 2) {
                                    w[u / 2] = bf16x2(v[u], v[u + 1]);
                                    v[u] -= __uint_as_float(w[u / 2] << 16);
                                    v[u + 1] -= __uint_as_float(w[u / 2] & 0xffff0000u);
                                }
                                if (live) st_v8(dst + ((size_t)pl * p.ld_dl + k) * 2, w);
                            }
                        } else {
                            uint32_t w[8];
#pragma unroll
                            for (int u = 0; u < 16; u += 2) w[u / 2] = bf16x2(v[u], v[u + 1]);
                            if (live && c0 + k < g.N) st_v8(dst + 2 * k, w);
                        }
                    }
                } else if constexpr (EPI == kAcc) {
                    float *dst = p.acc + ((size_t)T.part * g.M + row) * p.ld_acc + c0;
#pragma unroll
                    for (int k = 0; k < 128; k += 8) {
                        if (!live || c0 + k >= g.N) break;  // ld_acc is a multiple of 8
                        if (p.acc_add) {
                            uint32_t o[8];
                            ld_v8(dst + k, o);
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                r[k + u] = __float_as_uint(__uint_as_float(r[k + u]) + __uint_as_float(o[u]));
                        }
                        st_v8(dst + k, &r[k]);
                    }
                } else if constexpr (F32) {
#pragma unroll
                    for (int k = 0; k < 128; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * mul);
                    float *dst = (float *)g.out + g.ldo * row + c0;
#pragma unroll
                    for (int k = 0; k < 128; k += 4) {
                        if (!live) break;
                        if (g.vec && c0 + k + 4 <= g.N) {
                            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (g.add) o = *reinterpret_cast<const float4 *>(dst + k);
                            o.x += __uint_as_float(r[k]);
                            o.y += __uint_as_float(r[k + 1]);
                            o.z += __uint_as_float(r[k + 2]);
                            o.w += __uint_as_float(r[k + 3]);
                            *reinterpret_cast<float4 *>(dst + k) = o;
                        } else {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                if (c0 + k + u < g.N)
                                    dst[k + u] = (g.add ? dst[k + u] : 0.f) + __uint_as_float(r[k + u]);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 128; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * mul);
                    __nv_bfloat16 *dst = (__nv_bfloat16 *)g.out + g.ldo * row + c0;
                    if (live) {
#pragma unroll
                        for (int k = 0; k < 128; k += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                w[u] = bf16x2(__uint_as_float(r[k + 2 * u]), __uint_as_float(r[k + 2 * u + 1]));
                            if (g.vec == 2 && c0 + k + 16 <= g.N) {
                                st_v8(dst + k, w);  // whole 32-byte sectors
                                continue;
                            }
#pragma unroll
                            for (int v = 0; v < 16; v += 8) {
                                if (g.vec && c0 + k + v + 8 <= g.N) {
                                    *reinterpret_cast<uint4 *>(dst + k + v) =
                                        make_uint4(w[v / 2], w[v / 2 + 1], w[v / 2 + 2], w[v / 2 + 3]);
                                } else {
#pragma unroll
                                    for (int u = 0; u < 8; ++u)
                                        if (c0 + k + v + u < g.N)
                                            dst[k + v + u] = __float2bfloat16_rn(__uint_as_float(r[k + v + u]));
                                }
                            }
                        }
                    }
                }
            }
            if (EPI == kLse && live) p.part[((size_t)p.c0 + T.n0) / kTile * g.M + row] = make_float2(mx, l);
        }
        if (!ok) {
            atomicOr(p.err, kDevErrTimeout);
            *abort_flag = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
    }
}

template <int EPI, bool A_MN, bool B_MN, bool F32>
cudaError_t launch(const XentParams &p, const XentGemm &g, const CUtensorMap &a, const CUtensorMap &b,
                   cudaStream_t s) {
    constexpr auto kern = &xent_tc_kernel<EPI, A_MN, B_MN, F32>;
    cudaError_t e = allow_smem<kern>(kSmem);
    if (e != cudaSuccess) return e;
    const int tiles = g.mt * g.nt * g.parts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (tiles < g.pairs ? tiles : g.pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, b, p, g);
    return e != cudaSuccess ? e : cudaGetLastError();
}

int up(int a, int b) { return (a + b - 1) / b; }

// Rows of a box of A.
int box_rows(int rows) { return rows < 128 ? up(rows, 8) * 8 : 128; }

XentGemm shape(const XentParams &p, int M, int N, int K, int parts, int pairs) {
    XentGemm g{};
    g.M = M;
    g.N = N;
    g.K = K;
    g.mt = up(M, kTile);
    g.nt = up(N, kTile);
    g.parts = parts;
    g.k_part = parts > 1 ? up(up(K, parts), kBK) * kBK : up(K, kBK) * kBK;
    g.segments = p.planes == 3 ? 6 : 1;
    g.pairs = pairs;
    g.a_rows = box_rows(M);
    return g;
}

// A map of a row-major bf16 matrix of `planes` planes side by side: boxes of 64 x box_rows.
bool encode(CUtensorMap *m, const void *base, int width, int planes, long long plane, int rows, long long ld,
            int box_rows) {
    const long long all = planes > 1 ? planes * plane : width;
    const long long size[2] = {all, rows}, stride[1] = {rows > 1 ? ld : (all + 7) / 8 * 8};
    const int box[2] = {64, box_rows};
    return encode_bf16_map(m, base, 2, size, stride, box);
}
bool encode_x(CUtensorMap *m, const XentParams &p, int box_rows) {
    return encode(m, p.x, p.d, p.planes, p.plane_x, p.n, p.ldx, box_rows);
}
bool encode_w(CUtensorMap *m, const XentParams &p, int box_rows) {
    return encode(m, p.w, p.d, p.planes, p.plane_w, p.c1 - p.c0, p.ldw, box_rows);
}
bool encode_dl(CUtensorMap *m, const XentParams &p, int box_rows) {
    return encode(m, p.dl, p.c1 - p.c0, p.planes, p.ld_dl, p.n, p.planes * p.ld_dl, box_rows);
}
template <bool A_MN, bool B_MN>
cudaError_t launch_out(const XentParams &p, XentGemm &g, void *out, long long ldo, const CUtensorMap &a,
                       const CUtensorMap &b, cudaStream_t s) {
    g.out = out;
    g.ldo = ldo;
    const long long bytes = ldo * (p.planes == 3 ? 4 : 2);
    const uintptr_t at = reinterpret_cast<uintptr_t>(out);
    g.vec = bytes % 32 == 0 && at % 32 == 0 ? 2 : bytes % 16 == 0 && at % 16 == 0 ? 1 : 0;
    return p.planes == 3 ? launch<kOut, A_MN, B_MN, true>(p, g, a, b, s) : launch<kOut, A_MN, B_MN, false>(p, g, a, b, s);
}

}  // namespace

// The rows a TMA box can start on: base and row stride multiples of 16 bytes.
bool xent_tc_rows(const void *p, long long ld, int rows) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || (ld > 0 && ld % 8 == 0 && ld < 1ll << 36));
}

cudaError_t launch_xent_lse(const XentParams &p, int pairs, cudaStream_t s) {
    CUtensorMap a, b;
    if (!encode_x(&a, p, box_rows(p.n)) || !encode_w(&b, p, 128)) return cudaErrorInvalidValue;
    XentGemm g = shape(p, p.n, p.c1 - p.c0, p.d, 1, pairs);
    g.a_plane = p.plane_x;
    g.b_plane = p.plane_w;
    return p.planes == 3 ? launch<kLse, false, false, true>(p, g, a, b, s) : launch<kLse, false, false, false>(p, g, a, b, s);
}
cudaError_t launch_xent_dl(const XentParams &p, int pairs, cudaStream_t s) {
    CUtensorMap a, b;
    if (!encode_x(&a, p, box_rows(p.n)) || !encode_w(&b, p, 128)) return cudaErrorInvalidValue;
    XentGemm g = shape(p, p.n, p.c1 - p.c0, p.d, 1, pairs);
    g.a_plane = p.plane_x;
    g.b_plane = p.plane_w;
    return p.planes == 3 ? launch<kDl, false, false, true>(p, g, a, b, s) : launch<kDl, false, false, false>(p, g, a, b, s);
}
// dx (direct: the whole of it, written in its type; otherwise partial sums in acc)
cudaError_t launch_xent_dx(const XentParams &p, bool direct, int pairs, cudaStream_t s) {
    CUtensorMap a, b;
    if (!encode_dl(&a, p, box_rows(p.n)) || !encode_w(&b, p, 64)) return cudaErrorInvalidValue;
    XentGemm g = shape(p, p.n, p.d, p.c1 - p.c0, p.parts, pairs);
    g.a_plane = (int)p.ld_dl;
    g.b_plane = p.plane_w;
    if (direct) return launch_out<false, true>(p, g, p.dx, p.lddx, a, b, s);
    return p.planes == 3 ? launch<kAcc, false, true, true>(p, g, a, b, s) : launch<kAcc, false, true, false>(p, g, a, b, s);
}
// dw from the rows [r0, r1); add (fp32): onto what the rows before them gave
cudaError_t launch_xent_dw(const XentParams &whole, int r0, int r1, bool add, int pairs, cudaStream_t s) {
    CUtensorMap a, b;
    XentParams p = whole;
    p.n = r1 - r0;
    p.x = (const __nv_bfloat16 *)whole.x + whole.ldx * r0;
    p.dl = (__nv_bfloat16 *)whole.dl + (size_t)whole.planes * whole.ld_dl * r0;
    if (!encode_dl(&a, p, 64) || !encode_x(&b, p, 64)) return cudaErrorInvalidValue;
    XentGemm g = shape(p, p.c1 - p.c0, p.d, p.n, 1, pairs);
    g.add = add;
    g.a_plane = (int)p.ld_dl;
    g.b_plane = p.plane_x;
    return launch_out<true, true>(p, g, p.dw, p.lddw, a, b, s);
}

// CTA pairs that are resident at once on the current device.
cudaError_t xent_tc_pairs(int *pairs) {
    auto kern = xent_tc_kernel<kLse, false, false, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(148);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(pairs, kern, &cfg);
    if (e == cudaSuccess && *pairs < 1) e = cudaErrorInvalidConfiguration;
    return e;
}

}  // namespace fs
