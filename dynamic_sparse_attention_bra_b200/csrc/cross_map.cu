#include "cross_map.h"

namespace bra {

bool encode_heads_map(CUtensorMap* map, const void* base, int B, int L, int heads, int d, long long row,
                      long long batch, int box_tokens, int box_heads) {
    const EncodeTiledFn fn = tensor_map_encoder();
    const int box_c = d < 64 ? 32 : 64;
    if (!fn || d % box_c != 0 || box_tokens > 256 || box_heads > 256) return false;
    if (row <= 0 || row >= 1LL << 38 || batch < 0 || batch >= 1LL << 38) return false;
    if (batch == 0) {  // every entry has the same tokens
        B = 1;
        batch = row;
    }
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)row * 2, (cuuint64_t)batch * 2};
    const cuuint32_t box[4] = {(cuuint32_t)box_c, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, box_c == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace bra
