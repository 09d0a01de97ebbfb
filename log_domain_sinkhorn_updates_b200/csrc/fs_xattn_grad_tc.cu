// Gradient of cross attention on the sm_100a tensor cores, in two passes that
// each keep what they sum in TMEM (no atomics: the order of every sum is fixed):
//
//   KEYS  a CTA keeps 128 keys (K and V) and streams Q and dO in tiles of 64
//         queries over the heads that share the key head:
//           S^T = K Q^T, dP^T = V dO^T, P^T = 2^(S^T c + b_j - L_i), dS^T = P^T (dP^T - D_i)
//           dV += P^T dO, dK += dS^T Q
//   ROWS  a CTA keeps 128 packed rows (Q and dO) and streams K and V in tiles of 64 keys:
//           S = Q K^T, dP = dO V^T, P, dS as above, dQ += dS K
//
// In both the kept side is the left factor, so S, dP and with them P and dS
// come out with the kept rows in TMEM's lanes: they are written back as bf16
// (the type of the other operand, as in the forward) over the scores they came
// from and are the left factor of the next products there.  The streamed tile is
// the right factor of both kinds of product, once with its width and once with its
// rows as the K axis: the same shared-memory tile under two descriptors.  Seven
// products instead of the five of one combined pass, in exchange for sums that
// never leave the SM.
//
// Where there are fewer CTAs than SMs the streamed tiles are split into parts,
// whose raw sums a second kernel adds in their order.
//
// TMEM (512 columns): two or three buffers of S / P and dP / dS (64 columns
// each), the sums behind them.  Warps: 0 loads by TMA, 1 allocates TMEM, 1 and 3
// issue the MMAs of the scores and of the sums, 2 statistics, bias and masks,
// 4..7 and 8..11 turn scores into P and dS for even and odd tiles.
#include <cuda.h>

#include "fs_ops_tc.cuh"

namespace fs {
namespace {

using namespace tc;

constexpr int kTile = 64;  // streamed rows of a tile
constexpr int kThreads = 384;
constexpr int kColSlots = 4;

struct Layout {
    uint32_t st2, ring, half, cols, bars, total;
};
__host__ __device__ inline Layout layout(int atoms, int slots) {
    Layout L;
    L.st2 = (uint32_t)atoms * 16384u;
    L.ring = 2 * L.st2;
    L.half = (uint32_t)atoms * 8192u;
    L.cols = L.ring + (uint32_t)slots * 2u * L.half;
    L.bars = L.cols + kColSlots * 2 * kTile * 4;
    L.total = L.bars + (3 * slots + 2 * kColSlots + 2 + 3 + 3 + 3 + 2) * 8 + 32;
    return L;
}

// KS: steps of 16 along the widths (d and dv, the larger of the two), zeros beyond each.
template <bool KEYS, int KS>
__device__ void grad_pass(const CUtensorMap &map_q, const CUtensorMap &map_g, const CUtensorMap &map_k,
                          const CUtensorMap &map_v, const AttnParams &p, const AttnGradTc &g, int block, int part) {
    const CUtensorMap &map_s1 = KEYS ? map_q : map_k, &map_s2 = KEYS ? map_g : map_v;  // streamed
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    constexpr int kAtoms = (KS + 3) / 4;
    // Score buffers, 128 TMEM columns each (S / P, then dP / dS): as many as the sums leave room for.  With three, a
    // tile's scores wait for the sums of the tile three before it, not for those of its own group's last.
    constexpr int NB = KEYS && KS > 4 ? 2 : 3;
    constexpr uint32_t kSum1 = 128u * NB, kSum2 = kSum1 + (KS > 4 ? 128u : 64u);  // KEYS: dV, dK; ROWS: dQ
    const int NS = g.slots;
    const Layout L = layout(kAtoms, NS);
    uint8_t *st1 = smem, *st2 = smem + L.st2, *ring = smem + L.ring;
    float *sCols = reinterpret_cast<float *>(smem + L.cols);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L.bars);  // [NS] streamed tiles loaded
    uint64_t *ready = full + NS;                                   // [NS] masked rows cleared (ROWS)
    uint64_t *empty = ready + NS;                                  // [NS]
    uint64_t *cfull = empty + NS;                                  // [kColSlots]
    uint64_t *cempty = cfull + kColSlots;                          // [kColSlots]
    uint64_t *stfull = cempty + kColSlots;                         // kept side loaded
    uint64_t *stready = stfull + 1;                                // kept side usable
    uint64_t *sfull = stready + 1;                                 // [3]
    uint64_t *pready = sfull + 3;                                  // [3]
    uint64_t *pfree = pready + 3;                                  // [3]
    uint64_t *done = pfree + 3;                                    // every sum is complete
    uint64_t *sdone = done + 1;                                    // every score is
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sdone + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile int *tile_masked = reinterpret_cast<volatile int *>(tmem_holder + 2);  // [kColSlots]

    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int c = blockIdx.y % p.kv_heads, b = blockIdx.y / p.kv_heads;
    const int r0 = block * 128;  // first kept row (key, or packed query row)
    const int keys = attn_grad_keys(p, b), rows = p.n * p.group;
    const float top = p.top ? p.top[b] : 0.f;
    const int head_tiles = (p.n + kTile - 1) / kTile;
    const int all = KEYS ? (r0 < keys ? p.group * head_tiles : 0) : (keys + kTile - 1) / kTile;
    const int parts = KEYS ? p.key_parts : p.row_parts;
    const int t_beg = (int)((long long)all * part / parts), nt = (int)((long long)all * (part + 1) / parts) - t_beg;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full + s, 1);
            mbar_init(ready + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int s = 0; s < kColSlots; ++s) {
            mbar_init(cfull + s, 1);
            mbar_init(cempty + s, 4);
        }
        mbar_init(stfull, 1);
        mbar_init(stready, KEYS ? 1 : 8);
        for (int i = 0; i < 3; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(pready + i, 4);
            mbar_init(pfree + i, 1);
        }
        mbar_init(done, 1);
        mbar_init(sdone, 1);
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

    if (warp == 0) {
        // ---------------- loads ----------------
        if (lane == 0) {
            bool ok = true;
            if (KEYS && nt > 0) {  // the kept 128 keys, as two boxes of 64
                mbar_expect_tx(stfull, 2u * kAtoms * 16384u);
                for (int a = 0; a < kAtoms; ++a)
                    for (int u = 0; u < 2; ++u) {
                        tma_load_4d(saddr(st1) + a * 16384u + u * 8192u, &map_k, saddr(stfull), a * 64, r0 + 64 * u,
                                    c * g.k_head, b * g.k_batch);
                        tma_load_4d(saddr(st2) + a * 16384u + u * 8192u, &map_v, saddr(stfull), a * 64, r0 + 64 * u,
                                    c * g.v_head, b * g.v_batch);
                    }
            }
            int t = 0, y = (KEYS ? t_beg % head_tiles : t_beg) * kTile;
            int h = KEYS ? c * p.group + t_beg / head_tiles : c;
            RingPos rp{0, 0};
            for (; ok && t < nt; ++t) {
                const int s = rp.slot;
                if (*abort_flag) break;
                if (t >= NS && !mbar_wait_near(empty + s, rp.phase ^ 1u, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = saddr(ring + (size_t)s * 2 * L.half);
                mbar_expect_tx(full + s, 2u * L.half);
                for (int a = 0; a < kAtoms; ++a) {
                    tma_load_4d(dst + a * 8192u, &map_s1, saddr(full + s), a * 64, y, h * (KEYS ? g.q_head : g.k_head),
                                b * (KEYS ? g.q_batch : g.k_batch));
                    tma_load_4d(dst + L.half + a * 8192u, &map_s2, saddr(full + s), a * 64, y,
                                h * (KEYS ? g.g_head : g.v_head), b * (KEYS ? g.g_batch : g.v_batch));
                }
                rp.step(1, NS);
                y += kTile;
                if (KEYS && y >= p.n) {
                    y = 0;
                    ++h;
                }
            }
            if (!ok) {
                atomicOr(p.err, kDevErrTimeout);
                *abort_flag = 1;
            }
            if (KEYS && nt > 0) mbar_wait_near(stfull, 0, p.timeout_ns);
            for (int k = max(0, t - NS); k < t; ++k)
                mbar_wait_near(full + (k % NS), (uint32_t)(k / NS) & 1u, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------- per-column terms of the streamed tiles, and masked keys ----------------
        bool ok = true;
        if (KEYS && nt > 0) {
            unsigned dead[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                dead[u] = __ballot_sync(~0u, attn_masked(p, b, r0 + 32 * u + lane, keys));
            if (!warp_all(mbar_wait_near(stfull, 0, p.timeout_ns))) ok = false;
            if (dead[0] | dead[1] | dead[2] | dead[3]) {
                clear_rows<128>(st1, kAtoms, dead, lane);
                clear_rows<128>(st2, kAtoms, dead, lane);
                fence_async();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(stready);
        }
        RingPos rp{0, 0};
        int i0 = t_beg % head_tiles * kTile, h = c * p.group + t_beg / head_tiles;  // KEYS: of the next tile
        // KEYS: -L (base 2) and -D of a query; one without a key, or past the end, gives P = 0.  ROWS: a key's bias.
        float n0[2], n1[2] = {0.f, 0.f};  // read a tile ahead
        auto fetch = [&](int t) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (KEYS) {
                    const int i = i0 + 32 * u + lane;
                    n0[u] = -INFINITY;
                    n1[u] = 0.f;
                    if (t < nt && i < p.n) {
                        const size_t at = ((size_t)b * p.heads + h) * p.n + i;
                        n0[u] = p.lse2[at];
                        n1[u] = p.dot[at];
                    }
                } else {
                    n0[u] = attn_bias2(p, b, (t_beg + t) * kTile + 32 * u + lane, keys, top);
                }
            }
            i0 += kTile;
            if (KEYS && i0 >= p.n) {
                i0 = 0;
                ++h;
            }
        };
        fetch(0);
        for (int t = 0; ok && t < nt; ++t) {
            const int j = t % kColSlots;
            float *col = sCols + j * 2 * kTile;
            float v0[2], v1[2];
            unsigned dead[2] = {0u, 0u};
            bool any = !KEYS && p.bias != nullptr;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                v0[u] = KEYS ? (n0[u] == -INFINITY ? -INFINITY : -n0[u]) : n0[u];
                v1[u] = -n1[u];
                if (!KEYS) {
                    dead[u] = __ballot_sync(~0u, v0[u] == -INFINITY);
                    any = any || dead[u];
                }
            }
            fetch(t + 1);
            if (t >= kColSlots &&
                !warp_all(mbar_wait_near(cempty + j, ((uint32_t)(t / kColSlots) & 1u) ^ 1u, p.timeout_ns)))
                ok = false;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                col[32 * u + lane] = v0[u];
                col[kTile + 32 * u + lane] = v1[u];
            }
            if (lane == 0) tile_masked[j] = any;
            __syncwarp();
            if (lane == 0) mbar_arrive(cfull + j);
            if (!KEYS) {
                const int s = rp.slot;
                if (!warp_all(mbar_wait_near(full + s, rp.phase, p.timeout_ns))) ok = false;
                rp.step(1, NS);
                if (dead[0] | dead[1]) {
                    uint8_t *tile = ring + (size_t)s * 2 * L.half;
                    clear_rows<kTile>(tile, kAtoms, dead, lane);
                    clear_rows<kTile>(tile + L.half, kAtoms, dead, lane);
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
    } else if (warp < 4) {
        // ---------------- MMA issuers: warp 1 the scores, warp 3 the sums ----------------
        // (converged warps: elect_lane; with one warp for both, a tile's scores waited behind the last tile's sums)
        const bool lead = elect_lane();
        const uint32_t idesc_s = make_idesc<0, 128, kTile>();
        const uint32_t idesc_1 = idesc_mn(KEYS ? g.dv_pad : g.d_pad), idesc_2 = idesc_mn(g.d_pad);
        const uint64_t a1 = make_sdesc(saddr(st1), 128u), a2 = make_sdesc(saddr(st2), 128u);
        const uint64_t r1 = make_sdesc(saddr(ring), 128u), r2 = make_sdesc(saddr(ring) + L.half, 128u);
        const uint64_t c1 = sdesc_mn(saddr(ring), 8192u), c2 = sdesc_mn(saddr(ring) + L.half, 8192u);
        const uint32_t slot16 = 2 * L.half >> 4;
        bool ok = nt == 0 || warp_all(mbar_wait_near(stready, 0, p.timeout_ns));
        RingPos sp{0, 0}, bp{0, 0};  // the next tile's slot and buffer (each warp counts its own)
        // S and dP of tile t into its buffers, once the products that read them last are complete
        auto scores = [&](int t) {
            const int u = bp.slot;
            if (!warp_all((t < NB || mbar_wait_near(pfree + u, bp.phase ^ 1u, p.timeout_ns)) &&
                          mbar_wait_near((KEYS ? full : ready) + sp.slot, sp.phase, p.timeout_ns)))
                return false;
            tc_fence_after();
            if (lead) {
                const uint64_t b1 = r1 + (uint64_t)(sp.slot * slot16), b2 = r2 + (uint64_t)(sp.slot * slot16);
                const uint32_t ts = tmem_base + 128u * u;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    tc_mma<0>(ts, a1 + (uint64_t)((k / 4) * 1024 + (k % 4) * 2),
                              b1 + (uint64_t)((k / 4) * 512 + (k % 4) * 2), idesc_s, k > 0 ? 1u : 0u);
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    tc_mma<0>(ts + 64u, a2 + (uint64_t)((k / 4) * 1024 + (k % 4) * 2),
                              b2 + (uint64_t)((k / 4) * 512 + (k % 4) * 2), idesc_s, k > 0 ? 1u : 0u);
                tc_commit(saddr(sfull + u));
            }
            __syncwarp();
            sp.step(1, NS);
            bp.step(1, NB);
            return true;
        };
        // the sums over tile t's streamed rows, once its P and dS are written
        auto sums = [&](int t) {
            const int u = bp.slot, xs = sp.slot;
            const bool aborted = *abort_flag;  // read under the wait
            if (!warp_all(mbar_wait_near(pready + u, bp.phase, p.timeout_ns) && !aborted)) return false;
            tc_fence_after();
            if (lead) {
                const uint64_t m1 = c1 + (uint64_t)(xs * slot16), m2 = c2 + (uint64_t)(xs * slot16);
                const uint32_t ts = tmem_base + 128u * u;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k) {
                    if (KEYS)
                        tc_mma_ts(tmem_base + kSum1, ts + 8u * k, m2 + (uint64_t)(k * 128), idesc_1,
                                  t > 0 || k > 0 ? 1u : 0u);
                    else
                        tc_mma_ts(tmem_base + kSum1, ts + 64u + 8u * k, m1 + (uint64_t)(k * 128), idesc_1,
                                  t > 0 || k > 0 ? 1u : 0u);
                }
                if (KEYS) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc_mma_ts(tmem_base + kSum2, ts + 64u + 8u * k, m1 + (uint64_t)(k * 128), idesc_2,
                                  t > 0 || k > 0 ? 1u : 0u);
                }
                tc_commit(saddr(pfree + u));
                tc_commit(saddr(empty + xs));
            }
            __syncwarp();
            sp.step(1, NS);
            bp.step(1, NB);
            return true;
        };
        if (warp == 1)
            for (int t = 0; ok && t < nt; ++t) ok = scores(t);
        else
            for (int t = 0; ok && t < nt; ++t) ok = sums(t);
        uint64_t *drain = warp == 1 ? sdone : done;
        if (lead) {
            if (!ok) {
                atomicOr(p.err, kDevErrTimeout);
                *abort_flag = 1;
            }
            tc_commit(saddr(drain));
        }
        __syncwarp();
        mbar_wait_near(drain, 0, p.timeout_ns);
    } else {
        // ---------------- P and dS ----------------
        const int q = warp & 3, grp = (warp - 4) >> 2;
        const int row = r0 + q * 32 + lane;
        float nl = 0.f, nd = 0.f;  // KEYS: the key's bias; ROWS: -L (base 2) and -D of the row
        if (KEYS) {
            nl = attn_bias2(p, b, row, keys, top);
        } else {
            const int tid = (int)threadIdx.x - 128;
            stage_packed<kAtoms>(st1, p.q, p.qs, p, b, c, r0, 128, p.d, tid, 256);
            stage_packed<kAtoms>(st2, p.dout, p.dos, p, b, c, r0, 128, p.dv, tid, 256);
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(stready);
            nl = -INFINITY;
            if (row < rows) {
                const size_t at = ((size_t)b * p.heads + c * p.group + row % p.group) * p.n + row / p.group;
                const float l = p.lse2[at];
                nl = l == -INFINITY ? -INFINITY : -l;
                nd = -p.dot[at];
            }
        }
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        RingPos bp{grp, 0};  // this group's next buffer
        const uint64_t cc = pack2(p.scale2, p.scale2), nl2 = pack2(nl, nl), nd2 = pack2(nd, nd);
        bool ok = true;
        for (int t = grp; t < nt; t += 2) {
            const int j = t % kColSlots, u = bp.slot;
            const uint32_t ts = tmem_base + lanes + 128u * u, td = ts + 64u;
            const bool aborted = *abort_flag;  // read under the waits
            if (!warp_all(mbar_wait_near(sfull + u, bp.phase, p.timeout_ns) &&
                          mbar_wait_near(cfull + j, (uint32_t)(t / kColSlots) & 1u, p.timeout_ns) && !aborted)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float4 *c0 = reinterpret_cast<const float4 *>(sCols + j * 2 * kTile);
            const bool masked = KEYS || tile_masked[j];
            uint32_t sr[2][32], dr[2][32];
            tmem_ld32(ts, sr[0]);
            tmem_ld32(td, dr[0]);
            tmem_ld_wait();
            tmem_ld32(ts + 32u, sr[1]);  // the second half arrives under the first one's arithmetic
            tmem_ld32(td + 32u, dr[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1) tmem_ld_wait();
                const uint32_t(&s)[32] = sr[h], (&d)[32] = dr[h];
                uint32_t wp[16], ws[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    uint64_t z0 = nl2, z1 = nl2, e0 = nd2, e1 = nd2;
                    if (masked) {
                        const float4 v = c0[8 * h + k / 4];
                        z0 = add2(z0, pack2(v.x, v.y));
                        z1 = add2(z1, pack2(v.z, v.w));
                    }
                    if (KEYS) {
                        const float4 v = c0[kTile / 4 + 8 * h + k / 4];
                        e0 = pack2(v.x, v.y);
                        e1 = pack2(v.z, v.w);
                    }
                    float p0, p1, p2, p3, g0, g1, g2, g3;
                    unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), cc, z0), p0, p1);
                    unpack2(fma2(pack2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), cc, z1), p2, p3);
                    p0 = ex2_approx(p0);
                    p1 = ex2_approx(p1);
                    p2 = ex2_approx(p2);
                    p3 = ex2_approx(p3);
                    unpack2(add2(pack2(__uint_as_float(d[k]), __uint_as_float(d[k + 1])), e0), g0, g1);
                    unpack2(add2(pack2(__uint_as_float(d[k + 2]), __uint_as_float(d[k + 3])), e1), g2, g3);
                    wp[k / 2] = bf16x2(p0, p1);
                    wp[k / 2 + 1] = bf16x2(p2, p3);
                    ws[k / 2] = bf16x2(p0 * g0, p1 * g1);
                    ws[k / 2 + 1] = bf16x2(p2 * g2, p3 * g3);
                }
                if (KEYS) tmem_st16(ts + 16u * h, wp);
                tmem_st16(td + 16u * h, ws);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(pready + u);
                mbar_arrive(cempty + j);
            }
            bp.step(2, NB);
        }
        if (ok && nt > 0 && !warp_all(mbar_wait_near(done, 0, p.timeout_ns))) ok = false;
        if (!ok) {
            atomicOr(p.err, kDevErrTimeout);
            *abort_flag = 1;
        }
        tc_fence_after();
        // KEYS: group 0 writes dv, group 1 dk.  ROWS: alternate 32-column pieces of dq.
        const bool second = KEYS && grp == 1;
        const int width = KEYS && grp == 0 ? p.dv : p.d;
        const float mul = KEYS && grp == 0 ? 1.f : p.scale;
        __nv_bfloat16 *dst;
        bool live;
        if (KEYS) {
            live = row < p.m;
            const fs_view &v = second ? p.dks : p.dvs;
            dst = (__nv_bfloat16 *)(second ? p.dk : p.dv_out) + v.batch * b + v.token * row + v.head * c;
        } else {
            live = row < rows;
            dst = (__nv_bfloat16 *)p.dq + p.dqs.batch * b + p.dqs.token * (row / p.group) +
                  p.dqs.head * (c * p.group + row % p.group);
        }
        const uint32_t to = tmem_base + lanes + (second ? kSum2 : kSum1);
        // a key that takes no part gets zeros, whatever stands in a query or its gradient
        const bool zero = nt == 0 || (KEYS && nl == -INFINITY);
        if (parts > 1) {  // a part: its raw sums
            float *base = KEYS ? (second ? p.part_dk : p.part_dv) : p.part_dq;
            const size_t padded = (size_t)(KEYS ? g.key_blocks : g.row_blocks) * 128;
            float *raw = base + (((size_t)part * gridDim.y + blockIdx.y) * padded + row) * width;
            for (int k = KEYS ? 0 : 32 * grp; k < width; k += KEYS ? 32 : 64) {
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld32(to + k, o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int u = 0; u < 32; u += 4)
                    if (live && k + u < width)
                        *reinterpret_cast<uint4 *>(raw + k + u) =
                            zero ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
            }
        } else {
            for (int k = KEYS ? 0 : 32 * grp; k < width; k += KEYS ? 32 : 64) {
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld32(to + k, o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int u = 0; u < 32; u += 8) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (!zero) {
                        w.x = bf16x2(__uint_as_float(o[u]) * mul, __uint_as_float(o[u + 1]) * mul);
                        w.y = bf16x2(__uint_as_float(o[u + 2]) * mul, __uint_as_float(o[u + 3]) * mul);
                        w.z = bf16x2(__uint_as_float(o[u + 4]) * mul, __uint_as_float(o[u + 5]) * mul);
                        w.w = bf16x2(__uint_as_float(o[u + 6]) * mul, __uint_as_float(o[u + 7]) * mul);
                    }
                    if (live && k + u < width) *reinterpret_cast<uint4 *>(dst + k + u) = w;  // widths: multiples of 8
                }
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

// Both passes in one launch: the CTAs of the second fill in behind the first's last wave.
template <int KS>
__global__ void __launch_bounds__(kThreads, 1)
    xattn_grad_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_g,
                         const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const AttnParams p, const AttnGradTc g) {
    grid_dependency_wait();
    const int x = blockIdx.x, keys = g.key_blocks * p.key_parts;
    if (x < keys)
        grad_pass<true, KS>(map_q, map_g, map_k, map_v, p, g, x / p.key_parts, x % p.key_parts);
    else
        grad_pass<false, KS>(map_q, map_g, map_k, map_v, p, g, (x - keys) / p.row_parts, (x - keys) % p.row_parts);
}

// Adds the parts' sums in their order, eight elements a thread: dk and dv of every key, then dq of every row.
__global__ void __launch_bounds__(256) xattn_grad_join_kernel(const AttnParams p, int key_padded, int row_padded) {
    const int d8 = p.d / 8, v8 = p.dv / 8, rows = p.n * p.group, hb = blockIdx.y, heads = gridDim.y;
    const int c = hb % p.kv_heads, b = hb / p.kv_heads;
    const unsigned e = blockIdx.x * 256u + threadIdx.x;
    const unsigned keys = p.key_parts > 1 ? (unsigned)p.m * (d8 + v8) : 0u;
    grid_dependency_wait();
    const float *part;
    __nv_bfloat16 *dst;
    int row, k, parts, padded, width;
    float mul = p.scale;
    if (e < keys) {
        row = (int)(e / (unsigned)(d8 + v8));
        k = (int)(e % (unsigned)(d8 + v8));
        const bool value = k >= d8;
        k = (value ? k - d8 : k) * 8;
        const fs_view &s = value ? p.dvs : p.dks;
        part = value ? p.part_dv : p.part_dk;
        dst = (__nv_bfloat16 *)(value ? p.dv_out : p.dk) + s.batch * b + s.token * row + s.head * c + k;
        width = value ? p.dv : p.d;
        if (value) mul = 1.f;
        parts = p.key_parts;
        padded = key_padded;
    } else {
        row = (int)((e - keys) / (unsigned)d8);
        k = (int)((e - keys) % (unsigned)d8) * 8;
        if (p.row_parts == 1 || row >= rows) return;
        part = p.part_dq;
        dst = (__nv_bfloat16 *)p.dq + p.dqs.batch * b + p.dqs.token * (row / p.group) +
              p.dqs.head * (c * p.group + row % p.group) + k;
        width = p.d;
        parts = p.row_parts;
        padded = row_padded;
    }
    const float4 *src = reinterpret_cast<const float4 *>(part + ((size_t)hb * padded + row) * width + k);
    const size_t step = (size_t)heads * padded * width / 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float4 u = src[i * step], v = src[i * step + 1];
        x.x += u.x, x.y += u.y, x.z += u.z, x.w += u.w;
        y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(bf16x2(x.x * mul, x.y * mul), bf16x2(x.z * mul, x.w * mul),
                                                 bf16x2(y.x * mul, y.y * mul), bf16x2(y.z * mul, y.w * mul));
}

template <int KS>
cudaError_t launch(const AttnParams &p, AttnGradTc g, const CUtensorMap &mq, const CUtensorMap &mg,
                   const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s) {
    constexpr int atoms = (KS + 3) / 4;
    const uint32_t limit = 227u * 1024u;
    g.slots = 8;
    while (layout(atoms, g.slots).total + 1024u > limit) --g.slots;
    const uint32_t need = layout(atoms, g.slots).total + 1024u;
    // at least half the shared memory: a CTA holds all of TMEM, so two on one SM would wait for each other
    const uint32_t smem = need > limit / 2 + 1024u ? need : limit / 2 + 1024u;
    constexpr auto kern = &xattn_grad_tc_kernel<KS>;
    cudaError_t e = allow_smem<kern>(limit);
    if (e != cudaSuccess) return e;
    g.key_blocks = (p.m + 127) / 128;
    g.row_blocks = (p.n * p.group + 127) / 128;
    return launch_dependent(kern, dim3(g.key_blocks * p.key_parts + g.row_blocks * p.row_parts, p.batch * p.kv_heads),
                            kThreads, smem, s, mq, mg, mk, mv, p, g);
}

}  // namespace

cudaError_t launch_xattn_grad_tc(const AttnParams &p, cudaStream_t s) {
    AttnGradTc g{};
    g.d_pad = (p.d + 15) / 16 * 16;
    g.dv_pad = (p.dv + 15) / 16 * 16;
    CUtensorMap mq, mg, mk, mv;
    if (!attn_map(&mq, p.q, p.qs, p.d, p.n, p.heads, p.batch, kTile, &g.q_head, &g.q_batch) ||
        !attn_map(&mg, p.dout, p.dos, p.dv, p.n, p.heads, p.batch, kTile, &g.g_head, &g.g_batch) ||
        !attn_map(&mk, p.k, p.ks, p.d, p.m, p.kv_heads, p.batch, kTile, &g.k_head, &g.k_batch) ||
        !attn_map(&mv, p.v, p.vs, p.dv, p.m, p.kv_heads, p.batch, kTile, &g.v_head, &g.v_batch))
        return cudaErrorInvalidValue;
    const int w = p.d > p.dv ? p.d : p.dv;
    if (w <= 32) return launch<2>(p, g, mq, mg, mk, mv, s);
    if (w <= 64) return launch<4>(p, g, mq, mg, mk, mv, s);
    if (w <= 96) return launch<6>(p, g, mq, mg, mk, mv, s);
    return launch<8>(p, g, mq, mg, mk, mv, s);
}

cudaError_t launch_xattn_grad_join(const AttnParams &p, cudaStream_t s) {
    const int rows = p.n * p.group, d8 = p.d / 8;
    const unsigned long long work = (p.key_parts > 1 ? (unsigned long long)p.m * (d8 + p.dv / 8) : 0ull) +
                                    (p.row_parts > 1 ? (unsigned long long)rows * d8 : 0ull);
    return launch_dependent(xattn_grad_join_kernel, dim3((unsigned)((work + 255) / 256), p.batch * p.kv_heads), 256, 0,
                            s, p, (p.m + 127) / 128 * 128, (rows + 127) / 128 * 128);
}

}  // namespace fs
