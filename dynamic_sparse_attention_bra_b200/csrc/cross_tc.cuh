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

}  // namespace cross
}  // namespace bra
