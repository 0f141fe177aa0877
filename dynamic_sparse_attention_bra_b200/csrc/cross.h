// Cross attention to an encoder's states: geometry and launchers (internal).
#pragma once

#include <atomic>
#include <cstddef>

#include "../../include/bra.h"
#include "common.cuh"

namespace bra {

// One call's geometry.  The query heads of a state head form its group (rep
// of them); the group's rows are numbered r = t * rep + (head in the group),
// so that the rows of one token are consecutive in memory.
struct CrossGeom {
    int B, Lq, Lk, heads, kv_heads, rep, d;
    int rows;  // rep * Lq
    float scale;
    long long q_row, q_batch, k_row, k_batch, v_row, v_batch;  // strides in elements
    const int32_t* kv_len;   // [B] or null
    const uint8_t* kv_mask;  // [B, Lk] or null
};

// Valid states of entry b: kv_len clamped to [0, Lk] (the mask not counted).
__device__ __forceinline__ int cross_len(const CrossGeom& g, int b) {
    if (!g.kv_len) return g.Lk;
    const int n = g.kv_len[b];
    return n < 0 ? 0 : (n > g.Lk ? g.Lk : n);
}
// Element offsets of row r (see above) of entry b, state head j.
__device__ __forceinline__ size_t cross_q_offset(const CrossGeom& g, int b, int j, int r) {
    const int t = r / g.rep, hh = r - t * g.rep;
    return (size_t)b * g.q_batch + (size_t)t * g.q_row + (size_t)(j * g.rep + hh) * g.d;
}
// ... of O, dO and dQ, which are dense [B, Lq, heads, d].
__device__ __forceinline__ size_t cross_o_offset(const CrossGeom& g, int b, int j, int r) {
    const int t = r / g.rep, hh = r - t * g.rep;
    return (((size_t)b * g.Lq + t) * g.heads + (size_t)(j * g.rep + hh)) * g.d;
}
// ... of the log sums and D, [B, heads, Lq].
__device__ __forceinline__ size_t cross_lse_offset(const CrossGeom& g, int b, int j, int r) {
    const int t = r / g.rep, hh = r - t * g.rep;
    return ((size_t)b * g.heads + (size_t)(j * g.rep + hh)) * g.Lq + t;
}

// Allows ``kernel`` its dynamic shared memory, once for each device (a launch
// attribute; setting it on every call would cost as much as a third of a launch).
template <auto kernel>
inline bool allow_shared(uint32_t bytes) {
    static std::atomic<uint64_t> done[4];  // a bit for each of 256 devices
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (done[dev >> 6].load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return false;
    done[dev >> 6].fetch_or(bit, std::memory_order_release);
    return true;
}

// Partial results of a key split: rows x d unnormalised sums, then (maximum in
// powers of two, sum) pairs, for every (split, entry, state head, row).
struct CrossParts {
    float* o;
    float2* ml;
};

// The scores of a call: what the forms of the kernels are chosen by, besides a
// product's least size.
inline double cross_scores(const CrossGeom& g) { return (double)g.rows * g.Lk * g.kv_heads * g.B; }

// How a forward call is cut: by its sizes alone, so that the workspace's size
// follows from the shape.
struct CrossPlan {
    int splits;  // parts of the states, joined by a second kernel (1: none)
};
CrossPlan cross_forward_plan(const CrossGeom& g, bool bf16);
size_t cross_forward_part_rows(const CrossGeom& g, const CrossPlan& p);  // 0 without a split

bra_status cross_forward_bf16(const CrossGeom& g, const CrossPlan& p, const void* q, const void* k, const void* v,
                              void* o, float* lse, CrossParts parts, int* status, cudaStream_t stream);
// The form for few states (bf16).
bool cross_short_covers(const CrossGeom& g);
bra_status cross_forward_short(const CrossGeom& g, const void* q, const void* k, const void* v, void* o, float* lse,
                               cudaStream_t stream);
// The form for many rows (tcgen05); covers() says from how many on it is taken.
bool cross_tc_covers(const CrossGeom& g);
int cross_tc_rows(const CrossGeom& g);
bra_status cross_forward_tc(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o,
                            float* lse, CrossParts parts, int* status, cudaStream_t stream);
bra_status cross_forward_f32(const CrossGeom& g, const CrossPlan& p, const void* q, const void* k, const void* v,
                             void* o, float* lse, CrossParts parts, cudaStream_t stream);
// Joins the parts of a split into o and lse.
bra_status cross_join(const CrossGeom& g, int splits, bool bf16, CrossParts parts, void* o, float* lse,
                      cudaStream_t stream);

// Backward: splits of the rows in the dK, dV kernel, whose fp32 parts
// ([split][2][B, Lk, kv_heads, d]) a second kernel joins.
int cross_backward_splits(const CrossGeom& g, bool bf16);
bra_status cross_backward_bf16(const CrossGeom& g, int splits, const void* q, const void* k, const void* v,
                               const void* o, const float* lse, const void* grad_o, void* dq, void* dk, void* dv,
                               float* delta, float* parts, int* status, cudaStream_t stream);
bool cross_tc_backward_covers(const CrossGeom& g);
int cross_tc_backward_splits(const CrossGeom& g);
bra_status cross_backward_tc(const CrossGeom& g, int splits, const void* q, const void* k, const void* v,
                             const void* o, const float* lse, const void* grad_o, void* dq, void* dk, void* dv,
                             float* delta, float* parts, int* status, cudaStream_t stream);
bra_status cross_backward_f32(const CrossGeom& g, int splits, const void* q, const void* k, const void* v,
                              const void* o, const float* lse, const void* grad_o, void* dq, void* dk, void* dv,
                              float* delta, float* parts, cudaStream_t stream);
bra_status cross_backward_join(const CrossGeom& g, int splits, bool bf16, const float* parts, void* dk, void* dv,
                               cudaStream_t stream);

}  // namespace bra
