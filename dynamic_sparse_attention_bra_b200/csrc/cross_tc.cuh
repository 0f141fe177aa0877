// Operands of the tcgen05 cross-attention kernels in shared memory (swizzled
// tiles of D bf16 a row and their descriptors), and bounded waits.
#pragma once

#include "cross_tile.cuh"

namespace bra {
namespace cross {

constexpr uint32_t kWait = 1u << 22;

// Byte offset of 16-byte chunk c of row r in a tile of ``rows`` rows: 64-byte
// rows with the 64-byte swizzle at D = 32; 128-byte rows with the 128-byte
// swizzle otherwise, channels 64.. of D = 128 in a second panel.
template <int D>
__device__ __forceinline__ uint32_t op_offset(int r, int c, int rows) {
    if constexpr (D == 32) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Descriptor of a K-major operand (rows x D), and what its k-th 16 channels add
// to it (the address field counts 16 bytes).
template <int D>
__device__ __forceinline__ uint64_t k_major(uint32_t tile) {
    if constexpr (D == 32) return ptx::smem_desc(tile, 16, 512, ptx::kSwizzle64B);
    return ptx::smem_desc(tile, 16, 1024, ptx::kSwizzle128B);
}
template <int D>
__device__ __forceinline__ constexpr uint32_t k_step(int kk, int rows) {
    return D == 32 ? (uint32_t)kk * 2u : (uint32_t)((kk >> 2) * rows * 8 + (kk & 3) * 2);
}
// Descriptor of a tile whose rows are the inner axis (rows x D, channels the N
// axis), and what its k-th 16 rows add.
template <int D>
__device__ __forceinline__ uint64_t n_major(uint32_t tile, int rows) {
    if constexpr (D == 32) return ptx::smem_desc(tile, 16, 512, ptx::kSwizzle64B);
    return ptx::smem_desc(tile, rows * 128, 1024, ptx::kSwizzle128B);
}
template <int D>
__device__ __forceinline__ constexpr uint32_t n_step(int kk) { return (uint32_t)kk * (D == 32 ? 64u : 128u); }

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, int* abort, int* status) {
    for (uint32_t i = 0; i < kWait; ++i) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((i & 1023) == 1023 && *reinterpret_cast<volatile int*>(abort) != 0) return false;
    }
    *reinterpret_cast<volatile int*>(abort) = 1;
    raise_status(status, kDevTimeout);
    return false;
}

// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort, int* status) {
    if (__all_sync(0xffffffffu, ptx::mbar_test(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort, status));
}

// ``rows`` rows of queries (dense: O's layout) from row0; past the last: zeros.
template <int D>
__device__ __forceinline__ void tc_load_queries(uint32_t dst, const __nv_bfloat16* base, bool dense, const CrossGeom& g,
                                             int b, int j, int row0, int rows, int lane) {
#pragma unroll 4
    for (int e = lane; e < rows * (D / 8); e += 32) {
        const int r = e / (D / 8), c = e % (D / 8);
        const bool on = row0 + r < g.rows;
        const size_t off = !on ? 0 : dense ? cross_o_offset(g, b, j, row0 + r) : cross_q_offset(g, b, j, row0 + r);
        ptx::cp_async16_zfill(dst + op_offset<D>(r, c, rows), base + off + (on ? c * 8 : 0), on ? 16u : 0u);
    }
}

// ``rows`` rows of states from key0, those from ``end`` on not read.
template <int D>
__device__ __forceinline__ void tc_load_states(uint32_t dst, const __nv_bfloat16* base, long long step, int key0, int end,
                                            int rows, int lane) {
#pragma unroll 4
    for (int e = lane; e < rows * (D / 8); e += 32) {
        const int r = e / (D / 8), c = e % (D / 8);
        const bool on = key0 + r < end;
        ptx::cp_async16_zfill(dst + op_offset<D>(r, c, rows), on ? base + (size_t)(key0 + r) * step + c * 8 : base,
                              on ? 16u : 0u);
    }
}

// Validity of 32 W states from key0 as bits, the same in every lane of the warp.
template <int W>
__device__ __forceinline__ void valid_words(const CrossGeom& g, int b, int n, int key0, int lane, uint32_t (&w)[W]) {
#pragma unroll
    for (int h = 0; h < W; ++h) {
        const int left = n - key0 - h * 32;
        w[h] = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
    }
    if (g.kv_mask) {
        const uint8_t* m = g.kv_mask + (size_t)b * g.Lk + key0 + lane;
        uint8_t on[W];
#pragma unroll
        for (int h = 0; h < W; ++h) on[h] = (w[h] >> lane) & 1u ? __ldcg(m + h * 32) : (uint8_t)0;
#pragma unroll
        for (int h = 0; h < W; ++h) w[h] = __ballot_sync(0xffffffffu, on[h] != 0);
    }
}

// Zeros in the rows of TILES tiles (``second`` bytes apart; 32 W rows) whose bit
// in the W words is off.  A whole warp.
template <int D, int W, int TILES = 2>
__device__ __forceinline__ void clear_states(uint32_t dst, uint32_t second, const uint32_t* words, int lane) {
    constexpr int kPer = TILES * D / 8;  // 16-byte chunks of a row
#pragma unroll
    for (int h = 0; h < W; ++h) {
        const uint32_t w = words[h];
        if (w == 0xffffffffu) continue;
#pragma unroll 4
        for (int e = lane; e < 32 * kPer; e += 32) {
            const int r = e / kPer, c = e % kPer;
            if (!((w >> r) & 1u))
                ptx::st_shared_v4(dst + (c >= D / 8 ? second : 0u) + op_offset<D>(h * 32 + r, c % (D / 8), W * 32), 0u, 0u,
                                  0u, 0u);
        }
    }
}

}  // namespace cross
}  // namespace bra
