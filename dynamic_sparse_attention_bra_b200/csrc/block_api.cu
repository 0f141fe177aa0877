// C ABI of the operators around the attention in a conditioned block: cross
// attention to an encoder's states, rotary positions, dropout with the
// residual's sum.  Argument checks, workspace layout and launches; the
// contract of every entry point is in include/bra.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/bra.h"
#include "cross.h"
#include "rotary.h"

namespace bra {
namespace {

constexpr size_t kStatusBytes = 256;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// A required buffer: non-null and aligned, unless it has no elements.
bool buffer(const void* p, bool used) { return !used || (p && aligned16(p)); }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool known_dtype(int t) { return t == BRA_DTYPE_F32 || t == BRA_DTYPE_BF16; }
int vector_elems(int dtype) { return dtype == BRA_DTYPE_BF16 ? 8 : 4; }

// Strides of a [B, L, heads * d] operand: rows do not overlap, 16-byte steps.
bool good_strides(int64_t row, int64_t batch, int64_t width, int L, int vec) {
    if (row < 0 || batch < 0 || row % vec || batch % vec) return false;
    if (L > 1 && row < width) return false;
    return row <= (int64_t)1 << 40 && batch <= (int64_t)1 << 50;
}

bra_status make_cross(const bra_cross_shape* s, CrossGeom* g) {
    if (!s) return BRA_ERR_INVALID_ARG;
    if (s->B < 0 || s->Lq < 0 || s->Lk < 0 || s->heads <= 0 || s->kv_heads <= 0 || s->d <= 0)
        return BRA_ERR_INVALID_ARG;
    if (s->heads % s->kv_heads || !known_dtype(s->dtype)) return BRA_ERR_INVALID_ARG;
    // the kernels' exponents are powers of two: scale log2(e) is finite too
    if (!(s->scale > 0.f) || !std::isfinite(s->scale * 1.44269504f)) return BRA_ERR_INVALID_ARG;
    if (s->d != 32 && s->d != 64 && s->d != 128) return BRA_ERR_UNSUPPORTED;
    if (s->B > 65535 || s->heads > 1024 || s->Lk > 1 << 28 || (int64_t)s->Lq * s->heads > 1 << 28)
        return BRA_ERR_UNSUPPORTED;
    const int vec = vector_elems(s->dtype);
    const int64_t wq = (int64_t)s->heads * s->d, wk = (int64_t)s->kv_heads * s->d;
    if (!good_strides(s->q_row, s->q_batch, wq, s->Lq, vec) || !good_strides(s->k_row, s->k_batch, wk, s->Lk, vec) ||
        !good_strides(s->v_row, s->v_batch, wk, s->Lk, vec))
        return BRA_ERR_INVALID_ARG;
    g->B = s->B; g->Lq = s->Lq; g->Lk = s->Lk;
    g->heads = s->heads; g->kv_heads = s->kv_heads; g->d = s->d;
    g->rep = s->heads / s->kv_heads;
    g->rows = g->rep * s->Lq;
    g->scale = s->scale;
    g->q_row = s->q_row; g->q_batch = s->q_batch;
    g->k_row = s->k_row; g->k_batch = s->k_batch;
    g->v_row = s->v_row; g->v_batch = s->v_batch;
    g->kv_len = nullptr;
    g->kv_mask = nullptr;
    return BRA_OK;
}

// Workspace: status block | D of the backward | parts of a split (of the
// forward's states or the backward's rows, never both at a time).
struct CrossWorkspace {
    int* status;
    float* delta;
    float* parts;
    size_t bytes;
};

CrossWorkspace carve_cross(const CrossGeom& g, bool bf16, void* ws) {
    const size_t delta = round_up((size_t)g.B * g.heads * g.Lq * sizeof(float), 256);
    const size_t rows = cross_forward_part_rows(g, cross_forward_plan(g, bf16));
    const size_t fwd = rows * ((size_t)g.d + 2) * sizeof(float);
    const int sb = cross_backward_splits(g, bf16);
    const size_t bwd = sb > 1 ? (size_t)sb * 2 * g.B * g.Lk * g.kv_heads * g.d * sizeof(float) : 0;
    char* base = static_cast<char*>(ws);
    return {reinterpret_cast<int*>(base), reinterpret_cast<float*>(base + kStatusBytes),
            reinterpret_cast<float*>(base + kStatusBytes + delta),
            kStatusBytes + delta + round_up(fwd > bwd ? fwd : bwd, 256)};
}

bra_status make_rotary(const bra_rotary_shape* s, bool with_k, RotaryGeom* g) {
    if (!s) return BRA_ERR_INVALID_ARG;
    if (s->B < 0 || s->T < 0 || s->H < 0 || s->W < 0 || s->heads <= 0 || s->d <= 0 || !known_dtype(s->dtype))
        return BRA_ERR_INVALID_ARG;
    if (s->kv_heads < 0 || (with_k && s->kv_heads == 0)) return BRA_ERR_INVALID_ARG;
    int64_t pairs = 0;
    for (int a = 0; a < 3; ++a) {
        if (s->pairs[a] < 0) return BRA_ERR_INVALID_ARG;
        pairs += s->pairs[a];
    }
    if (pairs < 1 || 2 * pairs > s->d) return BRA_ERR_INVALID_ARG;
    if (s->d % 8 || s->d > 512 || s->B > 65535 || s->heads > 1024 || s->kv_heads > 1024) return BRA_ERR_UNSUPPORTED;
    const int64_t HW = (int64_t)s->H * s->W;
    if (HW > 1 << 28 || HW * s->T > 1 << 28) return BRA_ERR_UNSUPPORTED;
    const int L = (int)(HW * s->T), vec = vector_elems(s->dtype);
    const int64_t wq = (int64_t)s->heads * s->d, wk = (int64_t)s->kv_heads * s->d;
    if (!good_strides(s->q_row, s->q_batch, wq, L, vec) || !good_strides(s->qo_row, s->qo_batch, wq, L, vec) ||
        (s->B > 1 && s->qo_batch < wq))
        return BRA_ERR_INVALID_ARG;
    if (with_k && (!good_strides(s->k_row, s->k_batch, wk, L, vec) || !good_strides(s->ko_row, s->ko_batch, wk, L, vec) ||
                   (s->B > 1 && s->ko_batch < wk)))
        return BRA_ERR_INVALID_ARG;
    if (s->pos_batch < 0) return BRA_ERR_INVALID_ARG;
    g->B = s->B; g->L = L; g->H = s->H; g->W = s->W;
    g->heads = s->heads; g->kv_heads = with_k ? s->kv_heads : 0; g->d = s->d;
    g->P = (int)pairs; g->axis1 = s->pairs[0]; g->axis2 = s->pairs[0] + s->pairs[1];
    g->interleaved = s->interleaved != 0; g->inverse = s->inverse != 0;
    g->pos_batch = s->pos_batch;
    g->q_row = s->q_row; g->q_batch = s->q_batch; g->k_row = s->k_row; g->k_batch = s->k_batch;
    g->qo_row = s->qo_row; g->qo_batch = s->qo_batch; g->ko_row = s->ko_row; g->ko_batch = s->ko_batch;
    return BRA_OK;
}

}  // namespace
}  // namespace bra

using namespace bra;

extern "C" {

size_t bra_cross_workspace_bytes(const bra_cross_shape* shape) {
    CrossGeom g;
    if (make_cross(shape, &g) != BRA_OK) return 0;
    return carve_cross(g, shape->dtype == BRA_DTYPE_BF16, nullptr).bytes;
}

bra_status bra_cross_attend(const bra_cross_shape* shape, const void* q, const void* k, const void* v,
                            const int32_t* kv_len, const uint8_t* kv_mask, void* o, float* lse, void* workspace,
                            void* stream) {
    CrossGeom g;
    const bra_status rc = make_cross(shape, &g);
    if (rc != BRA_OK) return rc;
    const bool rows = g.B > 0 && g.Lq > 0, states = g.B > 0 && g.Lk > 0;
    if (!buffer(q, rows) || !buffer(o, rows) || !buffer(k, states) || !buffer(v, states) || !buffer(workspace, true) ||
        !aligned4(lse) || !aligned4(kv_len))
        return BRA_ERR_INVALID_ARG;
    if (!rows) return BRA_OK;
    g.kv_len = kv_len;
    g.kv_mask = kv_mask;
    const bool bf16 = shape->dtype == BRA_DTYPE_BF16;
    const CrossPlan p = cross_forward_plan(g, bf16);
    const CrossWorkspace w = carve_cross(g, bf16, workspace);
    const CrossParts parts{w.parts,
                           reinterpret_cast<float2*>(w.parts + cross_forward_part_rows(g, p) * (size_t)g.d)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return bf16 ? cross_forward_bf16(g, p, q, k, v, o, lse, parts, w.status, st)
                : cross_forward_f32(g, p, q, k, v, o, lse, parts, st);
}

bra_status bra_cross_attend_backward(const bra_cross_shape* shape, const void* q, const void* k, const void* v,
                                     const int32_t* kv_len, const uint8_t* kv_mask, const void* o, const float* lse,
                                     const void* grad_o, void* dq, void* dk, void* dv, void* workspace,
                                     void* stream) {
    CrossGeom g;
    const bra_status rc = make_cross(shape, &g);
    if (rc != BRA_OK) return rc;
    const bool rows = g.B > 0 && g.Lq > 0, states = g.B > 0 && g.Lk > 0;
    if (!buffer(q, rows) || !buffer(o, rows) || !buffer(lse, rows) || !buffer(grad_o, rows) || !buffer(dq, rows) ||
        !buffer(k, states) || !buffer(v, states) || !buffer(dk, states) || !buffer(dv, states) ||
        !buffer(workspace, true) || !aligned4(kv_len))
        return BRA_ERR_INVALID_ARG;
    const bool bf16 = shape->dtype == BRA_DTYPE_BF16;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!rows) {  // no query: the states' gradients are zero
        const size_t bytes = (size_t)g.B * g.Lk * g.kv_heads * g.d * (bf16 ? 2 : 4);
        if (bytes && (cudaMemsetAsync(dk, 0, bytes, st) != cudaSuccess ||
                      cudaMemsetAsync(dv, 0, bytes, st) != cudaSuccess))
            return BRA_ERR_CUDA;
        return BRA_OK;
    }
    g.kv_len = kv_len;
    g.kv_mask = kv_mask;
    const CrossWorkspace w = carve_cross(g, bf16, workspace);
    const int splits = cross_backward_splits(g, bf16);
    return bf16 ? cross_backward_bf16(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, w.delta, w.parts, w.status, st)
                : cross_backward_f32(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, w.delta, w.parts, st);
}

bra_status bra_cross_device_status(const bra_cross_shape* shape, void* workspace, void* stream) {
    CrossGeom g;
    const bra_status rc = make_cross(shape, &g);
    if (rc != BRA_OK) return rc;
    if (!workspace || !aligned16(workspace)) return BRA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int host = 0;
    if (cudaMemcpyAsync(&host, workspace, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess || cudaMemsetAsync(workspace, 0, sizeof(int), st) != cudaSuccess)
        return BRA_ERR_CUDA;
    return host == kDevOk ? BRA_OK : host == kDevTimeout ? BRA_ERR_TIMEOUT : BRA_ERR_CUDA;
}

bra_status bra_rotary(const bra_rotary_shape* shape, const void* q, const void* k, const int32_t* pos,
                      const float* inv_freq, void* q_out, void* k_out, void* stream) {
    RotaryGeom g;
    const bool with_k = k != nullptr || k_out != nullptr;
    const bra_status rc = make_rotary(shape, with_k, &g);
    if (rc != BRA_OK) return rc;
    const bool used = g.B > 0 && g.L > 0;
    if (!inv_freq || !aligned4(inv_freq) || !aligned4(pos)) return BRA_ERR_INVALID_ARG;
    if (!buffer(q, used) || !buffer(q_out, used) || (with_k && (!buffer(k, used) || !buffer(k_out, used))))
        return BRA_ERR_INVALID_ARG;
    // in place: the same rows are read and written
    if (used && q == q_out && (g.q_row != g.qo_row || g.q_batch != g.qo_batch)) return BRA_ERR_INVALID_ARG;
    if (used && with_k && k == k_out && (g.k_row != g.ko_row || g.k_batch != g.ko_batch)) return BRA_ERR_INVALID_ARG;
    if (!used) return BRA_OK;
    return rotary_launch(g, shape->dtype == BRA_DTYPE_BF16, q, k, pos, inv_freq, q_out, k_out,
                         static_cast<cudaStream_t>(stream));
}

bra_status bra_dropout_add(int dtype, int64_t n, int64_t unit, double p, const uint64_t* rng, const void* x,
                           const void* residual, void* y, void* stream) {
    if (!known_dtype(dtype) || n < 0 || unit < 1 || !(p >= 0.0 && p <= 1.0)) return BRA_ERR_INVALID_ARG;
    if (unit != 1 && unit % 8) return BRA_ERR_UNSUPPORTED;
    if (n > (int64_t)1 << 40) return BRA_ERR_UNSUPPORTED;
    if (!rng || (reinterpret_cast<uintptr_t>(rng) & 7u)) return BRA_ERR_INVALID_ARG;
    if (!buffer(x, n > 0) || !buffer(y, n > 0) || !aligned16(residual)) return BRA_ERR_INVALID_ARG;
    if (n == 0) return BRA_OK;
    const uint64_t threshold = (uint64_t)std::ceil(p * 4294967296.0);
    const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    return dropout_add_launch(dtype == BRA_DTYPE_BF16, n, unit, threshold, scale, rng, x, residual, y,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
