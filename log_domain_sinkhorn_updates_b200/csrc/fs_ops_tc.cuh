// Device helpers shared by the tensor-core kernels of the row-softmax operators.
#pragma once

#include "fs_ops.cuh"
#include "fs_tc_common.cuh"

namespace fs {
namespace tc {

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// mbar_wait that sleeps: one plain test (a phase that has completed costs no more), then the thread is suspended until
// the phase completes, or for 50 us a try.  Warps that wait then leave their issue slots to the softmax warp of the
// same SM quarter.
__device__ __forceinline__ bool mbar_done(uint64_t *b, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(done)
        : "r"(saddr(b)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool mbar_wait_near(uint64_t *b, uint32_t parity, unsigned long long limit_ns) {
    if (mbar_done(b, parity)) return true;
    unsigned long long t0 = 0;
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred P;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %3;\n\t"
            "selp.b32 %0, 1, 0, P;\n\t}"
            : "=r"(done)
            : "r"(saddr(b)), "r"(parity), "r"(50000u)
            : "memory");
        if (done) return true;
        const unsigned long long t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) return false;
    }
}
// What decides for a whole warp: every lane's answer.  A wait's time, or an abort flag, may run out for some lanes and not
// for others, and the barriers, votes, TMEM and MMA instructions that follow take all 32: without the vote a wait that
// ran out could leave part of a warp at one of them for good.
__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(~0u, ok); }
// A ring position that moves without divisions: slot and the parity of its use.
struct RingPos {
    int slot;
    uint32_t phase;
    __device__ __forceinline__ void step(int by, int slots) {
        slot += by;
        if (slot >= slots) {
            slot -= slots;
            phase ^= 1u;
        }
    }
};
// One lane of a converged warp.  A warp that issues MMAs runs its loop with all lanes, so that addresses and
// descriptors stay in uniform registers, and only the issuing instructions are one lane's: with the whole loop under
// lane == 0, each MMA took about 80 cycles to issue and a wait on a completed barrier 170 to 240.
__device__ __forceinline__ bool elect_lane() {
    uint32_t lead;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(lead));
    return lead != 0;
}
// The warpgroup gives up, or takes, registers: N a thread from here on.
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float max_of64(const uint32_t *s) {
    float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
    for (int k = 0; k < 64; k += 8) {
        t0 = max3(t0, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
        t1 = max3(t1, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
        t2 = max3(t2, __uint_as_float(s[k + 4]), __uint_as_float(s[k + 5]));
        t3 = max3(t3, __uint_as_float(s[k + 6]), __uint_as_float(s[k + 7]));
    }
    return fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
}
// A right factor as it lies in memory: its rows are the K axis, 64-element
// columns of its width `lbo` bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t addr, uint32_t lbo) {
    uint64_t desc = (uint64_t)((addr >> 4) & 0x3FFFu);
    desc |= (uint64_t)(lbo >> 4) << 16;
    desc |= (uint64_t)(1024u >> 4) << 32;
    desc |= (uint64_t)1u << 46;
    desc |= 2ull << 61;
    return desc;
}
// bf16 x bf16 -> fp32, M = 128, N columns, the right factor N-contiguous (sdesc_mn)
__device__ __forceinline__ uint32_t idesc_mn(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void group_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Packed rows [r0, r0 + count) (row r: query r / group, head c group + r % group) of a query-side bf16
// tensor of width w into 128-row blocks of ATOMS 64-element columns, as the 128-byte swizzle lays them; zeros
// beyond the last row and the width.  By threads t of `threads`.
template <int ATOMS>
__device__ __forceinline__ void stage_packed(uint8_t *dst, const void *src, const fs_view &s, const AttnParams &p, int b,
                                             int c, int r0, int count, int w, int t, int threads) {
    constexpr int per = ATOMS * 8;
    const int rows = p.n * p.group;
    for (int e = t; e < count * per; e += threads) {
        const int row = e / per, ch = e % per, at = r0 + row;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (at < rows && ch * 8 < w)
            v = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)src + s.batch * b + s.token * (at / p.group) +
                                                 s.head * (c * p.group + at % p.group) + ch * 8);
        *reinterpret_cast<uint4 *>(dst + (row >> 7) * ATOMS * 16384 + (ch >> 3) * 16384 + (row & 127) * 128 +
                                   (((ch & 7) ^ (row & 7)) << 4)) = v;
    }
}
// Zeroes the rows of a tile (ROWS x 64-element columns, `atoms` of them) whose bit of dead[row / 32] is set.  By one
// warp: a lane takes its rows whole (each starting at another piece, so that they lie in different banks), and a tile
// with few masked rows costs few stores.
template <int ROWS>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int atoms, const unsigned (&dead)[ROWS / 32], int lane) {
#pragma unroll
    for (int u = 0; u < ROWS / 32; ++u)
        if (dead[u] >> lane & 1u)
            for (int a = 0; a < atoms; ++a)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4 *>(tile + a * ROWS * 128 + (32 * u + lane) * 128 + ((k + lane) & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace tc
}  // namespace fs
