// Tensor maps of token operands [B, L, heads, d] with strides (host side).
#pragma once

#include "tma_host.h"

namespace bra {

// Tensor map of [B, L, heads, d] bf16 tokens with steps of ``row`` and ``batch``
// elements, whose box is box_tokens tokens of box_heads heads, 32 channels
// (64-byte swizzle) or 64 (128-byte swizzle) of each, landing as box_tokens x
// box_heads rows.  False too where a step does not fit a tensor map.
bool encode_heads_map(CUtensorMap* map, const void* base, int B, int L, int heads, int d, long long row,
                      long long batch, int box_tokens, int box_heads);

}  // namespace bra
