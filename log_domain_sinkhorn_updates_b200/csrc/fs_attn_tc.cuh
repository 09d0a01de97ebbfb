// Device helpers shared by the tensor-core cross-attention kernels.
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
// tensor of width w into 128-row blocks of `atoms` 64-element columns, as the 128-byte swizzle lays them; zeros
// beyond the last row and the width.  By threads t of `threads`.
__device__ __forceinline__ void stage_packed(uint8_t *dst, const void *src, const fs_view &s, const AttnParams &p, int b,
                                             int c, int r0, int count, int w, int atoms, int t, int threads) {
    const int per = atoms * 8, rows = p.n * p.group;
    for (int e = t; e < count * per; e += threads) {
        const int row = e / per, ch = e % per, at = r0 + row;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (at < rows && ch * 8 < w)
            v = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)src + s.batch * b + s.token * (at / p.group) +
                                                 s.head * (c * p.group + at % p.group) + ch * 8);
        *reinterpret_cast<uint4 *>(dst + (row >> 7) * atoms * 16384 + (ch >> 3) * 16384 + (row & 127) * 128 +
                                   (((ch & 7) ^ (row & 7)) << 4)) = v;
    }
}
// Zeroes the rows of a tile (`rows` x 64-element columns, `atoms` of them) whose bit of dead[row / 32] is set.
// By one warp.
__device__ __forceinline__ void clear_rows(uint8_t *tile, int rows, int atoms, const unsigned *dead, int lane) {
    for (int e = lane; e < rows * 8; e += 32) {
        const int row = e >> 3;
        unsigned word = dead[0];
        for (int u = 1; u < rows / 32; ++u)
            if (row / 32 == u) word = dead[u];
        if (word >> (row & 31) & 1u)
            for (int a = 0; a < atoms; ++a)
                *reinterpret_cast<uint4 *>(tile + a * rows * 128 + row * 128 + (e & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace tc
}  // namespace fs
