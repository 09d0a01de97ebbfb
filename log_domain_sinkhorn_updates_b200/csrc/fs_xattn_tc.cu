// Cross attention forward on the sm_100a tensor cores: S = Q K^T and O += P V
// per 64 keys with S, P and O in TMEM, one pass over the keys with a running
// maximum and sum a row.  Tiles of K and V: 128 keys (QT = 2) or 64 (QT = 1).
//
// A CTA has 128-row blocks of Q (rows r = query x heads that share the key
// head) and two softmax groups of 128 threads, a thread a row:
//  * QT = 2: two row blocks, each group its own, every K and V tile serves both
//    (whole sequences: half the stream of K and V a score);
//  * QT = 1: one row block, the groups take alternate key tiles into their own
//    S and O and are joined at the end (few rows; the loads of one tile run
//    under the softmax of the other).
// TMEM (512 columns): two buffers of 64 keys' scores a group, S_g / P_g in
// [128 g + 64 h, +64), O_g behind them in [256 + 128 g, ...).  While a group
// turns one buffer into weights, the products of the other and its next scores
// run: with one 128-key buffer, softmax, P V and the next S were a chain.
// P is written over the S it came from and is the A operand of the P V product
// there, in bf16 as V is (both operands of the product have one type; rounding
// either to more bits would take tf32, at half the rate and twice the bytes); V
// is its right factor as it lies in memory (width contiguous), by the descriptor.
//
// The maximum is lazy: the weights of 64 keys are taken against the running
// reference as it stands, and only where their sum passes 2^12 (which any score
// more than 12 above it forces, and infinity or NaN too), or at a row's first
// key, does the row move to those keys' maximum, O and the sum with it (by the
// row's own thread, between two products).  P stays below 2^12, exact to bf16's
// relative rounding as ever, and the common case spends nothing on the maximum
// and touches O from the tensor core alone.
//
// Keys past the length or masked by the bias: one warp reads the bias ahead,
// and where a tile has such keys it clears their rows of K and V in shared
// memory before the products read them, so that whatever stood there (NaN
// included) is a zero score plus -inf and a zero weight times zero.
//
// Warps: 0 loads K and V by TMA; 1 allocates TMEM; 1 and 2 issue the MMAs of
// groups 0 and 1; 3 bias and masks; 4..7 and 8..11 are the softmax groups.
#include <cuda.h>

#include "fs_ops_tc.cuh"

namespace fs {
namespace {

using namespace tc;

constexpr int kStep = 64;       // keys of a score buffer
constexpr int kThreads = 384;
constexpr int kBiasSlots = 4;
// Registers a thread of the 128 that load and issue, and of the 256 of the softmax: together the launch's 384 x 168.
constexpr int kFewRegs = 88, kManyRegs = 208;

// s = s c + bias over 64 scores (base 2)
__device__ __forceinline__ void add_bias(uint32_t (&s)[64], const float *bias, float c) {
    const float4 *bq = reinterpret_cast<const float4 *>(bias);
    const uint64_t cc = pack2(c, c);
#pragma unroll
    for (int k = 0; k < 64; k += 4) {
        const float4 bb = bq[k / 4];
        float z0, z1, z2, z3;
        unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), cc, pack2(bb.x, bb.y)), z0, z1);
        unpack2(fma2(pack2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), cc, pack2(bb.z, bb.w)), z2, z3);
        s[k] = __float_as_uint(z0);
        s[k + 1] = __float_as_uint(z1);
        s[k + 2] = __float_as_uint(z2);
        s[k + 3] = __float_as_uint(z3);
    }
}
// w = 2^(s mul - ref) as pairs of bf16, and the sum of the unrounded weights
__device__ __forceinline__ float weights(const uint32_t (&s)[64], float mul, float ref, uint32_t (&w)[32]) {
    const uint64_t cc = pack2(mul, mul), rn = pack2(-ref, -ref);
    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
    for (int k = 0; k < 64; k += 2) {
        float d0, d1;
        unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), cc, rn), d0, d1);
        d0 = ex2_approx(d0);
        d1 = ex2_approx(d1);
        acc[(k / 2) & 1] = add2(acc[(k / 2) & 1], pack2(d0, d1));
        w[k / 2] = bf16x2(d0, d1);
    }
    float a0, a1, a2, a3;
    unpack2(acc[0], a0, a1);
    unpack2(acc[1], a2, a3);
    return (a0 + a1) + (a2 + a3);
}

struct Layout {
    uint32_t q, ring, slot, bias, ml, bars, total;
};
// Keys of a loaded tile: two steps where both groups read it, one where each tile is one group's (what a group works
// on stays in the ring, and with 128 keys only a fifth of it was left for loads in flight: 111 us for 131072 keys
// of 8 heads).
__host__ __device__ constexpr int tile_keys(int qt) { return qt == 2 ? 128 : 64; }
__host__ __device__ inline Layout layout(int qt, int datoms, int vatoms, int slots) {
    Layout L;
    L.q = 0;
    L.ring = L.q + (uint32_t)qt * datoms * 16384u;
    L.slot = (uint32_t)((datoms > vatoms ? datoms : vatoms) * tile_keys(qt) * 128);
    L.bias = L.ring + (uint32_t)slots * L.slot;
    L.ml = L.bias + (uint32_t)(kBiasSlots * tile_keys(qt) * 4);
    L.bars = L.ml + 128 * 8;
    L.total = L.bars + (3 * slots + 2 * kBiasSlots + 1 + 4 + 4 + 4 + 2) * 8 + 16;
    return L;
}

// KS: steps of 16 along d, fixed at compile time (descriptor offsets are then
// immediates); what lies beyond d is zero in shared memory.
template <int QT, int KS, bool LENGTHS>
__global__ void __launch_bounds__(kThreads, 1)
    xattn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const AttnParams p, const AttnTc g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    constexpr int kTS = tile_keys(QT), kSteps = kTS / kStep;
    constexpr uint32_t kAtom = kTS * 128;  // bytes of a tile's 64-element column
    const int NS = g.slots;
    const Layout L = layout(QT, g.datoms, g.vatoms, NS);
    uint8_t *sQ = smem + L.q, *ring = smem + L.ring;
    float *sBias = reinterpret_cast<float *>(smem + L.bias);
    float2 *sML = reinterpret_cast<float2 *>(smem + L.ml);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L.bars);  // [NS] tile loaded
    uint64_t *ready = full + NS;                                   // [NS] masked rows cleared
    uint64_t *empty = ready + NS;                                  // [NS] products that read it are complete
    uint64_t *bfull = empty + NS;                                  // [kBiasSlots]
    uint64_t *bempty = bfull + kBiasSlots;                         // [kBiasSlots]
    uint64_t *qfull = bempty + kBiasSlots;
    uint64_t *sfull = qfull + 1;    // [2][2] S of group g, buffer h
    uint64_t *pready = sfull + 4;   // [2][2] P is written over it
    uint64_t *pvdone = pready + 4;  // [2][2] the products that read P are complete
    uint64_t *drain = pvdone + 4;   // [2] every MMA of issuer g is complete
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    float *top_holder = reinterpret_cast<float *>(tmem_holder + 2);

    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rows = p.n * p.group;
    const AttnUnit unit = attn_unit<LENGTHS>(p);
    const int c = unit.c, b = unit.b, j_beg = unit.j_beg, j_end = unit.j_end;
    const int most = j_end > j_beg ? (j_end - j_beg + kTS - 1) / kTS : 0;
    // tiles whose scores take a bias from shared memory: all, or only the one that the keys end in
    auto masked_tile = [&](int t) { return p.bias != nullptr || j_beg + (t + 1) * kTS > j_end; };

    const float top = attn_top<kThreads>(p, b, j_beg, j_end, reinterpret_cast<float *>(sML));
    if (attn_stats_done(p, unit, top)) return;
    if (threadIdx.x == 0) {
        *top_holder = top;  // read again by the warps that need it
        for (int s = 0; s < NS; ++s) {
            mbar_init(full + s, 1);
            mbar_init(ready + s, 1);
            mbar_init(empty + s, QT);
        }
        for (int s = 0; s < kBiasSlots; ++s) {
            mbar_init(bfull + s, 1);
            mbar_init(bempty + s, 4 * QT);
        }
        mbar_init(qfull, 8);
        for (int i = 0; i < 4; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(pready + i, 4);
            mbar_init(pvdone + i, 1);
        }
        mbar_init(drain, 1);
        mbar_init(drain + 1, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_holder)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    const int nt = *top_holder == -INFINITY ? 0 : most;
    if (warp < 4) {
        regs_dec<kFewRegs>();
        if (warp == 0) {
            // ---------------- K and V tiles: slot 2 t holds K(t), slot 2 t + 1 V(t) ----------------
            if (lane == 0) {
                bool ok = true;
                RingPos rp{0, 0};
                int i = 0;
                for (; ok && i < 2 * nt; ++i) {
                    const int s = rp.slot;
                    if (*abort_flag) break;
                    if (i >= NS && !mbar_wait_near(empty + s, rp.phase ^ 1u, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const int atoms = i & 1 ? g.vatoms : g.datoms;
                    const CUtensorMap *map = i & 1 ? &map_v : &map_k;
                    const int hm = i & 1 ? g.v_head : g.k_head, bm = i & 1 ? g.v_batch : g.k_batch;
                    const uint32_t dst = saddr(ring + (size_t)s * L.slot);
                    mbar_expect_tx(full + s, (uint32_t)atoms * kAtom);
                    for (int a = 0; a < atoms; ++a)
                        tma_load_4d(dst + a * kAtom, map, saddr(full + s), a * 64, j_beg + (i >> 1) * kTS, c * hm,
                                    b * bm);
                    rp.step(1, NS);
                }
                if (!ok) {
                    atomicOr(p.err, kDevErrTimeout);
                    *abort_flag = 1;
                }
                for (int k = max(0, i - NS); k < i; ++k)
                    mbar_wait_near(full + (k % NS), (uint32_t)(k / NS) & 1u, p.timeout_ns);
            }
            __syncwarp();
        } else if (warp == 3) {
            // ---------------- bias slices and masked rows ----------------
            bool ok = true;
            RingPos rp{0, 0};
            RingPos bs{0, 0};
            int used = 0;
            const float from = *top_holder;
            float bv[kTS / 32], next[kTS / 32];  // base-2 bias of a tile's keys, read a tile ahead
#pragma unroll
            for (int u = 0; u < kTS / 32; ++u) next[u] = attn_bias2(p, b, j_beg + 32 * u + lane, j_end, from);
            for (int t = 0; ok && t < nt; ++t) {
                unsigned dead[kTS / 32], cleared = 0;
#pragma unroll
                for (int u = 0; u < kTS / 32; ++u) {
                    bv[u] = next[u];
                    next[u] = attn_bias2(p, b, j_beg + (t + 1) * kTS + 32 * u + lane, j_end, from);
                    dead[u] = __ballot_sync(~0u, bv[u] == -INFINITY);
                    cleared |= dead[u];
                }
                if (masked_tile(t)) {
                    if (used >= kBiasSlots && !warp_all(mbar_wait_near(bempty + bs.slot, bs.phase ^ 1u, p.timeout_ns)))
                        ok = false;
#pragma unroll
                    for (int u = 0; u < kTS / 32; ++u) sBias[bs.slot * kTS + 32 * u + lane] = bv[u];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bfull + bs.slot);
                    bs.step(1, kBiasSlots);
                    ++used;
                }
                for (int kv = 0; kv < 2; ++kv) {
                    const int s = rp.slot;
                    if (!warp_all(mbar_wait_near(full + s, rp.phase, p.timeout_ns))) ok = false;
                    rp.step(1, NS);
                    if (cleared) {
                        uint8_t *tile = ring + (size_t)s * L.slot;
                        clear_rows<kTS>(tile, kv ? g.vatoms : g.datoms, dead, lane);
                        fence_async();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(ready + s);
                }
                if (!warp_all(!*abort_flag)) break;
            }
            if (!ok && lane == 0) {
                atomicOr(p.err, kDevErrTimeout);
                *abort_flag = 1;
            }
            __syncwarp();
        } else {
            // ---------------- MMA issuers (warps 1 and 2, one a group) ----------------
            const bool lead = elect_lane();
            const int grp = warp - 1;
            const uint32_t idesc_s = make_idesc<0, 128, kStep>();
            const uint32_t idesc_o = idesc_mn(g.dv_pad);
            const uint64_t qd = make_sdesc(saddr(sQ) + (QT == 2 ? grp : 0) * g.datoms * 16384u, 128u);
            const uint64_t k0 = make_sdesc(saddr(ring), 128u), v0 = sdesc_mn(saddr(ring), kAtom);
            const uint32_t slot16 = L.slot >> 4;
            const uint32_t ts = tmem_base + (uint32_t)(grp * 128), to = ts + 256u;
            // this group's tiles: all of them, or those of its parity
            const int mine = QT == 2 ? nt : (nt - grp + 1) / 2, steps = kSteps * mine;
            constexpr int kNext = QT == 2 ? 2 : 4;  // slots from a tile of the group to its next
            RingPos kp{QT == 2 ? 0 : 2 * grp, 0}, vp{QT == 2 ? 1 : 2 * grp + 1, 0};
            // S of step i (part h of its tile) into buffer i & 1
            auto s_product = [&](int i) {
                const int h = i % kSteps, u = i & 1;
                if (h == 0 && !warp_all(mbar_wait_near(ready + kp.slot, kp.phase, p.timeout_ns))) return false;
                tc_fence_after();
                if (lead) {
                    const uint64_t kd = k0 + (uint64_t)(kp.slot * slot16 + h * 512);
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        tc_mma<0>(ts + 64u * u, qd + (uint64_t)((k / 4) * 1024 + (k % 4) * 2),
                                  kd + (uint64_t)((k / 4) * (kAtom / 16) + (k % 4) * 2), idesc_s, k > 0 ? 1u : 0u);
                    tc_commit(saddr(sfull + 2 * grp + u));
                    if (h == kSteps - 1) tc_commit(saddr(empty + kp.slot));
                }
                __syncwarp();
                if (h == kSteps - 1) kp.step(kNext, NS);
                return true;
            };
            bool ok = steps == 0 || warp_all(mbar_wait_near(qfull, 0, p.timeout_ns));
            for (int i = 0; ok && i < min(steps, 2); ++i) ok = s_product(i);
            for (int i = 0; ok && i < steps; ++i) {
                const int h = i % kSteps, u = i & 1;
                const uint32_t ph = (uint32_t)(i >> 1) & 1u;
                if (!warp_all((h != 0 || mbar_wait_near(ready + vp.slot, vp.phase, p.timeout_ns)) &&
                              mbar_wait_near(pready + 2 * grp + u, ph, p.timeout_ns) && !*abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lead) {
                    const uint64_t vd = v0 + (uint64_t)(vp.slot * slot16 + h * 512);
#pragma unroll
                    for (int k = 0; k < kStep / 16; ++k)  // 16 keys: 8 TMEM columns of P, 2048 bytes of V
                        tc_mma_ts(to, ts + 64u * u + 8u * k, vd + (uint64_t)(k * 128), idesc_o, i > 0 || k > 0 ? 1u : 0u);
                    tc_commit(saddr(pvdone + 2 * grp + u));
                    if (h == kSteps - 1) tc_commit(saddr(empty + vp.slot));
                }
                __syncwarp();
                if (h == kSteps - 1) vp.step(kNext, NS);
                // the S after next takes the columns of this P: not before the products that read it are complete (the
                // softmax has the other buffer's S meanwhile)
                if (i + 2 < steps) ok = warp_all(mbar_wait_near(pvdone + 2 * grp + u, ph, p.timeout_ns)) && s_product(i + 2);
            }
            if (lead) {
                if (!ok) {
                    atomicOr(p.err, kDevErrTimeout);
                    *abort_flag = 1;
                }
                tc_commit(saddr(drain + grp));
            }
            __syncwarp();
            mbar_wait_near(drain + grp, 0, p.timeout_ns);
            __syncwarp();
        }
    } else {
        // ---------------- softmax groups ----------------
        regs_inc<kManyRegs>();
        const int q = warp & 3, grp = (warp - 4) >> 2;
        const int rl = q * 32 + lane;
        const int blk = QT == 2 ? grp : 0;
        const int r = unit.r0 + blk * 128 + rl;  // packed row
        const bool warp_live = unit.r0 + blk * 128 + q * 32 < rows;
        // Q into shared memory, 16 bytes at a time, as the 128-byte swizzle lays it
        stage_packed<(KS + 3) / 4>(sQ, p.q, p.qs, p, b, c, unit.r0, QT * 128, p.d, (int)threadIdx.x - 128, 256);
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull);
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const uint32_t ts = tmem_base + lanes + (uint32_t)(grp * 128);
        const uint32_t to = tmem_base + lanes + 256u + (uint32_t)(grp * 128);
        const float c2 = p.scale2;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        int i = 0;  // steps of this group done
        for (int t = QT == 2 ? 0 : grp; ok && t < nt; t += QT == 2 ? 1 : 2) {
            const bool masked = masked_tile(t);
            const int j = masked && p.bias ? t % kBiasSlots : 0;
            if (masked &&
                !warp_all(mbar_wait_near(bfull + j, p.bias ? (uint32_t)(t / kBiasSlots) & 1u : 0u, p.timeout_ns))) {
                ok = false;
                break;
            }
#pragma unroll 1
            for (int h = 0; h < kSteps; ++h, ++i) {
                const int u = i & 1;
                if (!warp_all(mbar_wait_near(sfull + 2 * grp + u, (uint32_t)(i >> 1) & 1u, p.timeout_ns))) {
                    ok = false;
                    break;
                }
                if (warp_live) {
                    tc_fence_after();
                    uint32_t s[64], w[32];
                    tmem_ld32(ts + 64u * u, s);
                    tmem_ld32(ts + 64u * u + 32u, s + 32);
                    tmem_ld_wait();
                    float mul = c2;
                    if (masked) {  // scores in base 2 with the bias
                        add_bias(s, sBias + j * kTS + kStep * h, c2);
                        mul = 1.f;
                    }
                    float sum = weights(s, mul, m == -INFINITY ? 0.f : m, w);
                    const bool over = m == -INFINITY || !(sum <= kLazySum);
                    if (__any_sync(~0u, over)) {
                        // a first key, or one far above: the rows concerned move to the step's own maximum, O and the
                        // sum with them, once the products so far are complete
                        const float mn = over ? fmaxf(m, max_of64(s) * mul) : m;
                        if (i > 0) {
                            if (!warp_all(mbar_wait_near(pvdone + 2 * grp + (u ^ 1), (uint32_t)((i - 1) >> 1) & 1u,
                                                         p.timeout_ns))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
                            l *= f;
                            for (int k = 0; k < g.dv_pad; k += 16) {
                                uint32_t o[16];
                                tmem_ld16(to + k, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st16(to + k, o);
                            }
                        }
                        m = mn;
                        sum = weights(s, mul, m == -INFINITY ? 0.f : m, w);
                    }
                    l += sum;
                    tmem_st32(ts + 64u * u, w);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                }  // else no row of this warp exists: its lanes of P may hold anything
                if (lane == 0) mbar_arrive(pready + 2 * grp + u);
            }
            if (!ok) break;
            __syncwarp();
            if (masked && lane == 0) mbar_arrive(bempty + j);
        }
        if (ok && i > 0 &&
            !warp_all(mbar_wait_near(pvdone + 2 * grp + ((i - 1) & 1), (uint32_t)((i - 1) >> 1) & 1u, p.timeout_ns)))
            ok = false;
        if (!ok) {
            atomicOr(p.err, kDevErrTimeout);
            *abort_flag = 1;
        }
        tc_fence_after();
        float f0 = 1.f, f1 = 0.f;  // weights of this group's and the other group's sums
        float *xo = reinterpret_cast<float *>(ring);  // QT = 1: group 1's O, [column][row]
        if (QT == 1) {
            // every product has read the ring by now: each group has waited for its last one
            group_bar(1, 256);
            if (grp == 1) {
                sML[rl] = make_float2(m, l);
                if (warp_live && i > 0)
                    for (int k = 0; k < g.dv_pad; k += 16) {
                        uint32_t o[16];
                        tmem_ld16(to + k, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < 16; ++u) xo[(k + u) * 128 + rl] = __uint_as_float(o[u]);
                    }
            }
            group_bar(1, 256);
            if (grp == 0) {
                const float2 other = sML[rl];
                if (nt > 1) {
                    const float mn = fmaxf(m, other.x), ref = mn == -INFINITY ? 0.f : mn;
                    f0 = ex2_approx(m - ref);
                    f1 = ex2_approx(other.x - ref);
                    l = l * f0 + other.y * f1;
                    m = mn;
                }
            }
        }
        if (warp_live && (QT == 2 || grp == 0)) {
            const bool live = r < rows;
            if (!unit.whole) {
                const size_t at = unit.part + blk * 128 + rl;
                if (live) p.part_ml[at] = {*top_holder, m, l};
                if (nt > 0)
                    for (int k = 0; k < p.dv; k += 16) {
                        uint32_t o[16];
                        tmem_ld16(to + k, o);
                        tmem_ld_wait();
                        float v[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            v[u] = __uint_as_float(o[u]) * f0;
                            if (QT == 1 && nt > 1) v[u] = fmaf(xo[(k + u) * 128 + rl], f1, v[u]);
                        }
#pragma unroll
                        for (int u = 0; u < 16; u += 4)
                            if (live && k + u < p.dv)  // dv is a multiple of 8
                                *reinterpret_cast<float4 *>(p.part_o + at * p.dv + k + u) =
                                    make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
                    }
            } else if (p.stats) {
                if (live)
                    p.lse2[((size_t)b * p.heads + c * p.group + r % p.group) * p.n + r / p.group] =
                        (float)((double)m + log2((double)l));
            } else {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int h = c * p.group + r % p.group, i = r / p.group;
                __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out + p.os.batch * b + p.os.token * i + p.os.head * h;
                for (int k = 0; k < p.dv; k += 16) {
                    uint32_t o[16];
                    if (nt > 0) {
                        tmem_ld16(to + k, o);
                        tmem_ld_wait();
                    }
                    uint32_t w[8];
#pragma unroll
                    for (int u = 0; u < 16; u += 2) {
                        float v0 = 0.f, v1 = 0.f;
                        if (nt > 0) {
                            v0 = __uint_as_float(o[u]) * f0;
                            v1 = __uint_as_float(o[u + 1]) * f0;
                            if (QT == 1 && nt > 1) {
                                v0 = fmaf(xo[(k + u) * 128 + rl], f1, v0);
                                v1 = fmaf(xo[(k + u + 1) * 128 + rl], f1, v1);
                            }
                        }
                        w[u / 2] = bf16x2(v0 * inv, v1 * inv);
                    }
                    if (live) *reinterpret_cast<uint4 *>(dst + k) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (live && k + 8 < p.dv)
                        *reinterpret_cast<uint4 *>(dst + k + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
                if (p.lse && live)
                    p.lse[((size_t)b * p.heads + h) * p.n + i] =
                        l == 0.f ? -INFINITY : (float)(((double)m + log2((double)l)) * kLn2d + *top_holder);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
    }
}

template <int QT, int KS, bool LENGTHS>
cudaError_t launch(const AttnParams &p, AttnTc g, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s) {
    const uint32_t limit = 227u * 1024u;
    g.slots = QT == 2 ? 8 : 12;
    while (layout(QT, g.datoms, g.vatoms, g.slots).total + 1024u > limit) --g.slots;
    const uint32_t smem = layout(QT, g.datoms, g.vatoms, g.slots).total + 1024u;
    cudaError_t e = allow_smem<&xattn_tc_kernel<QT, KS, LENGTHS>>(limit);
    if (e != cudaSuccess) return e;
    // The softmax takes registers that the launch must have brought: a build with fewer would wait for them.
    static std::atomic<int> regs{0};
    if (regs == 0) {
        cudaFuncAttributes a{};
        e = cudaFuncGetAttributes(&a, xattn_tc_kernel<QT, KS, LENGTHS>);
        if (e != cudaSuccess) return e;
        regs = a.numRegs;
    }
    if (regs * kThreads < 128 * kFewRegs + 256 * kManyRegs) return cudaErrorInvalidConfiguration;
    // at least half the shared memory: a CTA holds all of TMEM, so two on one SM would wait for each other
    xattn_tc_kernel<QT, KS, LENGTHS><<<p.main_units + p.tail_units * p.splits, kThreads,
                              smem > limit / 2 + 1024u ? smem : limit / 2 + 1024u, s>>>(mk, mv, p, g);
    return cudaGetLastError();
}

template <bool LENGTHS>
cudaError_t launch_width(const AttnParams &p, const AttnTc &g, const CUtensorMap &mk, const CUtensorMap &mv,
                         cudaStream_t s) {
    const int ks = (p.d + 31) / 32 * 2;
    if (p.unit_rows == 256)
        return ks == 2   ? launch<2, 2, LENGTHS>(p, g, mk, mv, s)
               : ks == 4 ? launch<2, 4, LENGTHS>(p, g, mk, mv, s)
               : ks == 6 ? launch<2, 6, LENGTHS>(p, g, mk, mv, s)
                         : launch<2, 8, LENGTHS>(p, g, mk, mv, s);
    return ks == 2   ? launch<1, 2, LENGTHS>(p, g, mk, mv, s)
           : ks == 4 ? launch<1, 4, LENGTHS>(p, g, mk, mv, s)
           : ks == 6 ? launch<1, 6, LENGTHS>(p, g, mk, mv, s)
                     : launch<1, 8, LENGTHS>(p, g, mk, mv, s);
}

}  // namespace

// A [batch][token][head][w] bf16 tensor as a 4-D map (boxes of 64 x box_rows of one head); a head or batch axis of
// stride 0 or of one element is left out (*hm, *bm: what to multiply its index with).
bool attn_map(CUtensorMap *map, const void *base, const fs_view &s, int w, int tokens, int heads, int batch,
              int box_rows, int *hm, int *bm) {
    const long long unit = (w + 7) / 8 * 8;
    *hm = heads > 1 && s.head > 0 ? 1 : 0;
    *bm = batch > 1 && s.batch > 0 ? 1 : 0;
    const long long size[4] = {w, tokens, *hm ? heads : 1, *bm ? batch : 1};
    const long long stride[3] = {tokens > 1 ? s.token : unit, *hm ? s.head : unit, *bm ? s.batch : unit};
    const int box[4] = {64, box_rows, 1, 1};
    return encode_bf16_map(map, base, 4, size, stride, box);
}

// What the vector loads and the TMA boxes of the tensor-core kernels need of a tensor.
bool attn_tc_view(const void *base, const fs_view &s, int tokens, int heads, int batch, bool map) {
    const long long big = 1ll << 36;
    if (reinterpret_cast<uintptr_t>(base) & 15) return false;
    if (tokens > 1 && (s.token % 8 || s.token >= big || (map && s.token == 0))) return false;
    if (heads > 1 && (s.head % 8 || s.head >= big)) return false;
    return !(batch > 1 && (s.batch % 8 || s.batch >= big));
}

cudaError_t launch_xattn_tc(const AttnParams &p, cudaStream_t s) {
    const bool two_blocks = p.unit_rows == 256;
    AttnTc g{};
    g.datoms = (p.d + 63) / 64;
    g.vatoms = (p.dv + 63) / 64;
    g.dv_pad = (p.dv + 15) / 16 * 16;
    CUtensorMap mk, mv;
    const int box = tile_keys(two_blocks ? 2 : 1);
    if (!attn_map(&mk, p.k, p.ks, p.d, p.m, p.kv_heads, p.batch, box, &g.k_head, &g.k_batch) ||
        !attn_map(&mv, p.v, p.vs, p.dv, p.m, p.kv_heads, p.batch, box, &g.v_head, &g.v_batch))
        return cudaErrorInvalidValue;
    return p.k_len ? launch_width<true>(p, g, mk, mv, s) : launch_width<false>(p, g, mk, mv, s);
}

}  // namespace fs
