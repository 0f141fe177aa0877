// Rotary positions: geometry and launcher (internal).
#pragma once

#include "../../include/bra.h"
#include "common.cuh"

namespace bra {

struct RotaryGeom {
    int B, L, H, W;               // tokens; the grid's rows and columns (without given positions)
    int heads, kv_heads, d;       // kv_heads = 0: no K
    int P, axis1, axis2;          // pairs; first pair of height, of width
    int interleaved, inverse;
    long long pos_batch;          // elements between the entries' positions
    long long q_row, q_batch, k_row, k_batch, qo_row, qo_batch, ko_row, ko_batch;
};

bra_status rotary_launch(const RotaryGeom& g, bool bf16, const void* q, const void* k, const int32_t* pos,
                         const float* inv_freq, void* q_out, void* k_out, cudaStream_t stream);

// y = residual + (keep ? x * scale : 0), unit elements sharing a draw; keep = word >= threshold.
bra_status dropout_add_launch(bool bf16, int64_t n, int64_t unit, uint64_t threshold, float scale,
                              const uint64_t* rng, const void* x, const void* residual, void* y, cudaStream_t stream);

}  // namespace bra
