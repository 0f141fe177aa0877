// Tiles of the warp-MMA cross-attention kernels: 16-byte asynchronous loads
// of state or query rows into swizzled shared memory, the states' validity
// as bits, and the fragment loads of m16n8k16.
#pragma once

#include "cross.h"
#include "cross_ptx.cuh"
#include "warp_mma.cuh"

namespace bra {
namespace cross {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What a row's sum of 2^(s' - m) ends as: the factor of O, and the natural log sum.  Only a
// sum of zero is a row without valid states (O = 0, log sum -inf); a sum that is NaN,
// of a row with a score that is, stays NaN in both.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// The exponent's offset of a row: its log sum in powers of two; a row without
// valid states gets +inf, which makes its P zero.
__device__ __forceinline__ float exponent_offset(float lse) {
    return lse == -INFINITY ? INFINITY : lse * kLog2e;
}

// Byte offset of 16-byte chunk c of row r in a tile of D bf16 a row.  The
// chunk index is permuted so that the eight rows that one ldmatrix phase
// reads lie in distinct banks: two 64-byte rows share a 128-byte line at D = 32.
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
    if constexpr (D == 32)
        return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    else
        return (uint32_t)(r * (2 * D) + ((c ^ (r & 7)) << 4));
}

// Validity of states as bits, 32 a word.  Without a mask a word follows from
// the length alone; with one, words of 4096 states at a time are kept in
// shared memory (two such groups, since loads run ahead of the products).
struct ValidBits {
    static constexpr int kGroupTiles = 64, kWords = 128;
    uint32_t* smem;  // [2][kWords], used with a mask only
    const uint8_t* mask;
    int n;           // states below n exist

    // Called by the whole CTA before tile ``t`` (64 states) is first used;
    // fills the group of words that starts there.
    __device__ __forceinline__ void reach(int t, int first_tile, int threads) {
        if (!mask) return;
        if (t != first_tile && (t & (kGroupTiles - 1)) != 0) return;
        const int group = t / kGroupTiles;
        uint32_t* w = smem + (group & 1) * kWords;
        const int warps = threads >> 5, lane = threadIdx.x & 31;
        for (int i = threadIdx.x >> 5; i < kWords; i += warps) {
            const int key = group * 4096 + i * 32 + lane;
            const bool on = key < n && __ldcg(mask + key) != 0;
            const uint32_t b = __ballot_sync(0xffffffffu, on);
            if (lane == 0) w[i] = b;
        }
        __syncthreads();
    }
    __device__ __forceinline__ uint32_t word(int t, int half) const {
        if (mask) return smem[((t / kGroupTiles) & 1) * kWords + (t & (kGroupTiles - 1)) * 2 + half];
        const int left = n - (t * 64 + half * 32);
        return left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
    }
};

// 64 state rows of tile t: a row whose bit is off is filled with zeros and
// not read.
template <int D, int THREADS>
__device__ __forceinline__ void load_states(uint32_t dst, const __nv_bfloat16* base, long long row_stride, int t,
                                            uint32_t w0, uint32_t w1) {
    constexpr int kChunks = D / 8;
#pragma unroll
    for (int i = 0; i < 64 * kChunks / THREADS; ++i) {
        const int e = i * THREADS + (int)threadIdx.x, r = e / kChunks, c = e % kChunks;
        const bool on = ((r < 32 ? w0 : w1) >> (r & 31)) & 1u;
        const __nv_bfloat16* src = on ? base + (size_t)(t * 64 + r) * row_stride + c * 8 : base;
        ptx::cp_async16_zfill(dst + tile_offset<D>(r, c), src, on ? 16u : 0u);
    }
}

// B fragments of 16 columns (two n8 tiles) x 16 of the inner axis from a tile
// whose rows are the columns (scores: rows = states, inner axis = channels).
template <int D>
__device__ __forceinline__ void frag_nt(uint32_t tile, int row0, int kk, int lane, uint32_t (&b)[4]) {
    const int m = lane >> 3;
    wmma16::ldsm_x4(tile + tile_offset<D>(row0 + (m >> 1) * 8 + (lane & 7), kk * 2 + (m & 1)), b[0], b[1], b[2], b[3]);
}
// B fragments of 16 channels (two n8 tiles from chunk c) x 16 rows of the
// tile as the inner axis.
template <int D>
__device__ __forceinline__ void frag_nn(uint32_t tile, int row0, int c, int lane, uint32_t (&b)[4]) {
    const int m = lane >> 3;
    wmma16::ldsm_x4_t(tile + tile_offset<D>(row0 + (m & 1) * 8 + (lane & 7), c + (m >> 1)), b[0], b[1], b[2], b[3]);
}
// A fragment of 16 rows x 16 channels.
template <int D>
__device__ __forceinline__ void frag_a(uint32_t tile, int row0, int kk, int lane, uint32_t (&a)[4]) {
    const int m = lane >> 3;
    wmma16::ldsm_x4(tile + tile_offset<D>(row0 + (m & 1) * 8 + (lane & 7), kk * 2 + (m >> 1)), a[0], a[1], a[2], a[3]);
}

}  // namespace cross
}  // namespace bra
