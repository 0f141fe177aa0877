// Cross attention and its gradients in fp32, on CUDA cores (the formulas are
// those of the bf16 kernels; every product and sum is fp32).
//
// A CTA of 128 threads (16 x 8) owns a tile of rows and streams tiles of 64
// of the other side through shared memory.  A thread holds, of a product
// A B^T, the rows ty + 16 i and the columns tx + 8 c, and of an accumulation
// P B the same rows and the channels 4 tx + 32 c .. + 3; rows of a tile are
// padded by four floats, so that the eight rows a warp reads at a time lie in
// distinct banks.  FP32 multiply-adds bound it.
#include "cross_tile.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;

constexpr int kThreads = 128;
constexpr int kPRow = 68;

template <int D>
struct Tile {
    static constexpr int kRow = D + 4;
    static constexpr int kFloats = 64 * kRow;
};

template <int D>
__device__ __forceinline__ void load_states_f32(float* dst, const float* base, long long row_stride, int t,
                                                uint32_t w0, uint32_t w1) {
    constexpr int kChunks = D / 4;
    const uint32_t d = ptx::smem_addr(dst);
#pragma unroll
    for (int i = 0; i < 64 * kChunks / kThreads; ++i) {
        const int e = i * kThreads + (int)threadIdx.x, r = e / kChunks, c = e % kChunks;
        const bool on = ((r < 32 ? w0 : w1) >> (r & 31)) & 1u;
        ptx::cp_async16_zfill(d + (uint32_t)(r * Tile<D>::kRow + c * 4) * 4u,
                              on ? base + (size_t)(t * 64 + r) * row_stride + c * 4 : base, on ? 16u : 0u);
    }
}

template <int D, int ROWS>
__device__ __forceinline__ void load_rows_f32(float* dst, const float* base, const CrossGeom& g, int b, int j,
                                              int row0, bool dense) {
    constexpr int kChunks = D / 4;
    const uint32_t d = ptx::smem_addr(dst);
#pragma unroll
    for (int i = 0; i < ROWS * kChunks / kThreads; ++i) {
        const int e = i * kThreads + (int)threadIdx.x, r = e / kChunks, c = e % kChunks;
        const bool on = row0 + r < g.rows;
        const size_t off = !on ? 0 : dense ? cross_o_offset(g, b, j, row0 + r) : cross_q_offset(g, b, j, row0 + r);
        ptx::cp_async16_zfill(d + (uint32_t)(r * Tile<D>::kRow + c * 4) * 4u, base + off + (on ? c * 4 : 0),
                              on ? 16u : 0u);
    }
}

// s[i][c] = <A row ty + 16 i, B row tx + 8 c>
template <int D, int MR>
__device__ __forceinline__ void dot_tiles(const float* a, const float* b, int ty, int tx, float (&s)[MR][8]) {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) s[i][c] = 0.f;
#pragma unroll 4
    for (int x = 0; x < D; x += 4) {
        float4 av[MR];
#pragma unroll
        for (int i = 0; i < MR; ++i) av[i] = *reinterpret_cast<const float4*>(a + (ty + 16 * i) * Tile<D>::kRow + x);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float4 bv = *reinterpret_cast<const float4*>(b + (tx + 8 * c) * Tile<D>::kRow + x);
#pragma unroll
            for (int i = 0; i < MR; ++i) {
                s[i][c] = fmaf(av[i].x, bv.x, s[i][c]);
                s[i][c] = fmaf(av[i].y, bv.y, s[i][c]);
                s[i][c] = fmaf(av[i].z, bv.z, s[i][c]);
                s[i][c] = fmaf(av[i].w, bv.w, s[i][c]);
            }
        }
    }
}

// acc[i][c] += sum_k P[ty + 16 i][k] B[k][4 tx + 32 c ..]
template <int D, int MR>
__device__ __forceinline__ void accumulate_tiles(const float* p, const float* b, int ty, int tx,
                                                 float4 (&acc)[MR][D / 32]) {
#pragma unroll 4
    for (int k = 0; k < 64; k += 4) {
        float4 pv[MR];
#pragma unroll
        for (int i = 0; i < MR; ++i) pv[i] = *reinterpret_cast<const float4*>(p + (ty + 16 * i) * kPRow + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const float4 bv = *reinterpret_cast<const float4*>(b + (k + kk) * Tile<D>::kRow + 4 * tx + 32 * c);
#pragma unroll
                for (int i = 0; i < MR; ++i) {
                    const float w = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
                    acc[i][c].x = fmaf(w, bv.x, acc[i][c].x);
                    acc[i][c].y = fmaf(w, bv.y, acc[i][c].y);
                    acc[i][c].z = fmaf(w, bv.z, acc[i][c].z);
                    acc[i][c].w = fmaf(w, bv.w, acc[i][c].w);
                }
            }
    }
}

template <int MR, int N>
__device__ __forceinline__ void zero(float4 (&acc)[MR][N]) {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
}

template <int MR>
__device__ __forceinline__ void store_p(float* p, int ty, int tx, const float (&s)[MR][8]) {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) p[(ty + 16 * i) * kPRow + tx + 8 * c] = s[i][c];
}

// ------------------------------------------------------------------- forward
// MR rows a thread: 16 MR rows a CTA (MR = 1 for single tokens).
// shared memory: Q (16 MR rows) | K | V | P (16 MR rows) | mask bits
template <int D, int MR>
constexpr uint32_t fwd_smem() {
    return (uint32_t)(16 * MR * Tile<D>::kRow + 2 * Tile<D>::kFloats + 16 * MR * kPRow + 2 * ValidBits::kWords) * 4u;
}

template <int D, int MR>
__global__ void __launch_bounds__(kThreads)
bra_cross_f32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                     float* __restrict__ o, float* __restrict__ lse, CrossParts parts, CrossGeom g, int row_tiles,
                     int splits) {
    extern __shared__ __align__(16) float fs[];
    float* sq = fs;
    float* sk = sq + 16 * MR * Tile<D>::kRow;
    float* sv = sk + Tile<D>::kFloats;
    float* sp = sv + Tile<D>::kFloats;
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    int id = blockIdx.x;
    const int row0 = (id % row_tiles) * 16 * MR;
    id /= row_tiles;
    const int split = id % splits;
    id /= splits;
    const int j = id % g.kv_heads, b = id / g.kv_heads;
    grid_dependency_wait();
    const int n = cross_len(g, b), all = (n + 63) / 64, per = (all + splits - 1) / splits;
    const int t0 = split * per, t1 = min(all, t0 + per);
    ValidBits bits{reinterpret_cast<uint32_t*>(sp + 16 * MR * kPRow),
                   g.kv_mask ? g.kv_mask + (size_t)b * g.Lk : nullptr, n};
    load_rows_f32<D, 16 * MR>(sq, q, g, b, j, row0, false);
    const float c2 = g.scale * kLog2e;
    float4 acc[MR][D / 32];
    zero(acc);
    float m[MR], l[MR];
#pragma unroll
    for (int i = 0; i < MR; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    for (int t = t0; t < t1; ++t) {
        if (t > t0) __syncthreads();
        bits.reach(t, t0, kThreads);
        const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
        load_states_f32<D>(sk, k + (size_t)b * g.k_batch + (size_t)j * D, g.k_row, t, w0, w1);
        ptx::cp_async_commit();
        load_states_f32<D>(sv, v + (size_t)b * g.v_batch + (size_t)j * D, g.v_row, t, w0, w1);
        ptx::cp_async_commit();
        ptx::cp_async_wait_group<1>();
        __syncthreads();
        float s[MR][8];
        dot_tiles<D, MR>(sq, sk, ty, tx, s);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const bool on = ((c < 4 ? w0 : w1) >> ((tx + 8 * c) & 31)) & 1u;
#pragma unroll
            for (int i = 0; i < MR; ++i)
                if (!on) s[i][c] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < MR; ++i) {
            float mx = s[i][0];
#pragma unroll
            for (int c = 1; c < 8; ++c) mx = fmaxf(mx, s[i][c]);
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float mn = fmaxf(m[i], mx * c2), mu = mn == -INFINITY ? 0.f : mn;
            const float alpha = ptx::ex2(m[i] - mu);
            m[i] = mn;
            l[i] *= alpha;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                s[i][c] = ptx::ex2(fmaf(s[i][c], c2, -mu));
                l[i] += s[i][c];
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                acc[i][c].x *= alpha;
                acc[i][c].y *= alpha;
                acc[i][c].z *= alpha;
                acc[i][c].w *= alpha;
            }
        }
        store_p<MR>(sp, ty, tx, s);
        ptx::cp_async_wait_group<0>();
        __syncthreads();
        accumulate_tiles<D, MR>(sp, sv, ty, tx, acc);
    }
    ptx::cp_async_wait_all();
    allow_dependents();
#pragma unroll
    for (int i = 0; i < MR; ++i) {
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        const int r = row0 + ty + 16 * i;
        if (r >= g.rows) continue;
        if (splits > 1) {
            const size_t at = ((size_t)(split * g.B + b) * g.kv_heads + j) * g.rows + r;
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                *reinterpret_cast<float4*>(parts.o + at * D + 4 * tx + 32 * c) = acc[i][c];
            if (tx == 0) parts.ml[at] = make_float2(m[i], l[i]);
        } else {
            const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
            float* row = o + cross_o_offset(g, b, j, r);
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                *reinterpret_cast<float4*>(row + 4 * tx + 32 * c) =
                    make_float4(acc[i][c].x * inv, acc[i][c].y * inv, acc[i][c].z * inv, acc[i][c].w * inv);
            if (tx == 0 && lse)
                lse[cross_lse_offset(g, b, j, r)] = l[i] > 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
        }
    }
}

// ------------------------------------------------------------------ dQ and D
// shared memory: Q | dO | K | V | dS | D, log sums [64] | mask bits
template <int D>
constexpr uint32_t dq_smem() {
    return (uint32_t)(4 * Tile<D>::kFloats + 64 * kPRow + 128 + 2 * ValidBits::kWords) * 4u;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
bra_cross_f32_dq_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                        const float* __restrict__ o, const float* lse, const float* __restrict__ go,
                        float* __restrict__ dq, float* __restrict__ delta, CrossGeom g, int row_tiles) {
    extern __shared__ __align__(16) float fs[];
    float* sq = fs;
    float* sg = sq + Tile<D>::kFloats;
    float* sk = sg + Tile<D>::kFloats;
    float* sv = sk + Tile<D>::kFloats;
    float* sp = sv + Tile<D>::kFloats;
    float* sd = sp + 64 * kPRow;
    float* sl = sd + 64;
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    int id = blockIdx.x;
    const int row0 = (id % row_tiles) * 64;
    id /= row_tiles;
    const int j = id % g.kv_heads, b = id / g.kv_heads;
    grid_dependency_wait();
    const int n = cross_len(g, b), tiles = (n + 63) / 64;
    ValidBits bits{reinterpret_cast<uint32_t*>(sl + 64), g.kv_mask ? g.kv_mask + (size_t)b * g.Lk : nullptr, n};
    load_rows_f32<D, 64>(sq, q, g, b, j, row0, false);
    load_rows_f32<D, 64>(sg, go, g, b, j, row0, true);
    {
        const int r = threadIdx.x >> 1, half = threadIdx.x & 1;
        float x = 0.f;
        if (row0 + r < g.rows) {
            const size_t off = cross_o_offset(g, b, j, row0 + r) + half * (D / 2);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(o + off) + c);
                const float4 h = __ldcg(reinterpret_cast<const float4*>(go + off) + c);
                x = fmaf(f.x, h.x, x);
                x = fmaf(f.y, h.y, x);
                x = fmaf(f.z, h.z, x);
                x = fmaf(f.w, h.w, x);
            }
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        if (half == 0) {
            sd[r] = x;
            float ls = -INFINITY;
            if (row0 + r < g.rows) {
                const size_t at = cross_lse_offset(g, b, j, row0 + r);
                delta[at] = x;
                ls = __ldcg(lse + at);
            }
            sl[r] = exponent_offset(ls);
        }
    }
    const float c2 = g.scale * kLog2e;
    float4 acc[4][D / 32];
    zero(acc);
    for (int t = 0; t < tiles; ++t) {
        if (t > 0) __syncthreads();
        bits.reach(t, 0, kThreads);
        const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
        load_states_f32<D>(sk, k + (size_t)b * g.k_batch + (size_t)j * D, g.k_row, t, w0, w1);
        load_states_f32<D>(sv, v + (size_t)b * g.v_batch + (size_t)j * D, g.v_row, t, w0, w1);
        ptx::cp_async_wait_all();
        __syncthreads();
        float s[4][8], dp[4][8];
        dot_tiles<D, 4>(sq, sk, ty, tx, s);
        dot_tiles<D, 4>(sg, sv, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float dd = sd[ty + 16 * i], off = sl[ty + 16 * i];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const bool on = ((c < 4 ? w0 : w1) >> ((tx + 8 * c) & 31)) & 1u;
                s[i][c] = on ? ptx::ex2(fmaf(s[i][c], c2, -off)) * (dp[i][c] - dd) : 0.f;
            }
        }
        store_p<4>(sp, ty, tx, s);
        __syncthreads();
        accumulate_tiles<D, 4>(sp, sk, ty, tx, acc);
    }
    ptx::cp_async_wait_all();
    allow_dependents();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row0 + ty + 16 * i;
        if (r >= g.rows) continue;
        float* row = dq + cross_o_offset(g, b, j, r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            *reinterpret_cast<float4*>(row + 4 * tx + 32 * c) = make_float4(
                acc[i][c].x * g.scale, acc[i][c].y * g.scale, acc[i][c].z * g.scale, acc[i][c].w * g.scale);
    }
}

// -------------------------------------------------------------------- dK, dV
// shared memory: K | V | Q | dO | P^T | dS^T | log sums, D [64]
template <int D>
constexpr uint32_t dkv_smem() {
    return (uint32_t)(4 * Tile<D>::kFloats + 2 * 64 * kPRow + 128) * 4u;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
bra_cross_f32_dkv_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                         const float* lse, const float* __restrict__ go,
                         const float* delta, float* __restrict__ dk, float* __restrict__ dv,
                         float* __restrict__ parts, CrossGeom g, int key_tiles, int splits) {
    extern __shared__ __align__(16) float fs[];
    float* sk = fs;
    float* sv = sk + Tile<D>::kFloats;
    float* sq = sv + Tile<D>::kFloats;
    float* sg = sq + Tile<D>::kFloats;
    float* sp = sg + Tile<D>::kFloats;
    float* ss = sp + 64 * kPRow;
    float* sl = ss + 64 * kPRow;
    float* sd = sl + 64;
    const int lane = threadIdx.x & 31, tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    int id = blockIdx.x;
    const int kt = id % key_tiles;
    id /= key_tiles;
    const int split = id % splits;
    id /= splits;
    const int j = id % g.kv_heads, b = id / g.kv_heads;
    grid_dependency_wait();
    const int n = cross_len(g, b);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int key = kt * 64 + h * 32 + lane;
        const bool on = key < n && (!g.kv_mask || __ldcg(g.kv_mask + (size_t)b * g.Lk + key) != 0);
        w[h] = __ballot_sync(0xffffffffu, on);
    }
    const int all = (g.rows + 63) / 64, per = (all + splits - 1) / splits;
    const int t0 = split * per, t1 = (w[0] | w[1]) ? min(all, t0 + per) : t0;
    load_states_f32<D>(sk, k + (size_t)b * g.k_batch + (size_t)j * D, g.k_row, kt, w[0], w[1]);
    load_states_f32<D>(sv, v + (size_t)b * g.v_batch + (size_t)j * D, g.v_row, kt, w[0], w[1]);
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) on[i] = ((i < 2 ? w[0] : w[1]) >> ((ty + 16 * i) & 31)) & 1u;
    const float c2 = g.scale * kLog2e;
    float4 ak[4][D / 32], av[4][D / 32];
    zero(ak);
    zero(av);
    for (int t = t0; t < t1; ++t) {
        if (t > t0) __syncthreads();
        load_rows_f32<D, 64>(sq, q, g, b, j, t * 64, false);
        load_rows_f32<D, 64>(sg, go, g, b, j, t * 64, true);
        {
            const int r = threadIdx.x & 63;
            const bool in = t * 64 + r < g.rows;
            const size_t at = in ? cross_lse_offset(g, b, j, t * 64 + r) : 0;
            if (threadIdx.x < 64) sl[r] = in ? exponent_offset(__ldcg(lse + at)) : INFINITY;
            else sd[r] = in ? __ldcg(delta + at) : 0.f;
        }
        ptx::cp_async_wait_all();
        __syncthreads();
        float s[4][8], dp[4][8];
        dot_tiles<D, 4>(sk, sq, ty, tx, s);
        dot_tiles<D, 4>(sv, sg, ty, tx, dp);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float off = sl[tx + 8 * c], dd = sd[tx + 8 * c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i][c] = on[i] ? ptx::ex2(fmaf(s[i][c], c2, -off)) : 0.f;
                dp[i][c] = s[i][c] * (dp[i][c] - dd);
            }
        }
        store_p<4>(sp, ty, tx, s);
        store_p<4>(ss, ty, tx, dp);
        __syncthreads();
        accumulate_tiles<D, 4>(sp, sg, ty, tx, av);
        accumulate_tiles<D, 4>(ss, sq, ty, tx, ak);
    }
    ptx::cp_async_wait_all();
    allow_dependents();
    const size_t elems = (size_t)g.B * g.Lk * g.kv_heads * D;
    float* ok = splits > 1 ? parts + (size_t)split * 2 * elems : dk;
    float* ov = splits > 1 ? ok + elems : dv;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = kt * 64 + ty + 16 * i;
        if (key >= g.Lk) continue;
        const size_t at = (((size_t)b * g.Lk + key) * g.kv_heads + j) * D + 4 * tx;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            *reinterpret_cast<float4*>(ok + at + 32 * c) = make_float4(
                ak[i][c].x * g.scale, ak[i][c].y * g.scale, ak[i][c].z * g.scale, ak[i][c].w * g.scale);
            *reinterpret_cast<float4*>(ov + at + 32 * c) = av[i][c];
        }
    }
}

template <int D, int MR>
bra_status launch_forward(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o,
                          float* lse, CrossParts parts, cudaStream_t stream) {
    auto* kernel = bra_cross_f32_kernel<D, MR>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fwd_smem<D, MR>()) !=
        cudaSuccess)
        return BRA_ERR_CUDA;
    const int row_tiles = (g.rows + 16 * MR - 1) / (16 * MR);
    const long long grid = (long long)row_tiles * splits * g.kv_heads * g.B;
    if (grid > 0x7fffffffLL) return BRA_ERR_UNSUPPORTED;
    const cudaError_t e =
        launch_after_previous(kernel, dim3((unsigned)grid), dim3(kThreads), fwd_smem<D, MR>(), stream,
                              static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v),
                              static_cast<float*>(o), lse, parts, g, row_tiles, splits);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

template <int D>
bra_status forward_d(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o, float* lse,
                     CrossParts parts, cudaStream_t stream) {
    return g.rows <= 16 ? launch_forward<D, 1>(g, splits, q, k, v, o, lse, parts, stream)
                        : launch_forward<D, 4>(g, splits, q, k, v, o, lse, parts, stream);
}

template <int D>
bra_status backward_d(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, const void* o,
                      const float* lse, const void* go, void* dq, void* dk, void* dv, float* delta, float* parts,
                      cudaStream_t stream) {
    using T = float;
    if (cudaFuncSetAttribute(bra_cross_f32_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dq_smem<D>()) != cudaSuccess ||
        cudaFuncSetAttribute(bra_cross_f32_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dkv_smem<D>()) != cudaSuccess)
        return BRA_ERR_CUDA;
    const int row_tiles = (g.rows + 63) / 64, key_tiles = (g.Lk + 63) / 64;
    const long long grid_q = (long long)row_tiles * g.kv_heads * g.B;
    const long long grid_k = (long long)key_tiles * splits * g.kv_heads * g.B;
    if (grid_q > 0x7fffffffLL || grid_k > 0x7fffffffLL) return BRA_ERR_UNSUPPORTED;
    cudaError_t e = launch_after_previous(bra_cross_f32_dq_kernel<D>, dim3((unsigned)grid_q), dim3(kThreads),
                                          dq_smem<D>(), stream, (const T*)q, (const T*)k, (const T*)v, (const T*)o,
                                          lse, (const T*)go, (T*)dq, delta, g, row_tiles);
    if (e != cudaSuccess) return BRA_ERR_CUDA;
    if (grid_k == 0) return BRA_OK;
    e = launch_after_previous(bra_cross_f32_dkv_kernel<D>, dim3((unsigned)grid_k), dim3(kThreads), dkv_smem<D>(),
                              stream, (const T*)q, (const T*)k, (const T*)v, lse, (const T*)go, (const float*)delta,
                              (T*)dk, (T*)dv, parts, g, key_tiles, splits);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace

bra_status cross_forward_f32(const CrossGeom& g, const CrossPlan& p, const void* q, const void* k, const void* v,
                             void* o, float* lse, CrossParts parts, cudaStream_t stream) {
    const bra_status rc = g.d == 32   ? forward_d<32>(g, p.splits, q, k, v, o, lse, parts, stream)
                          : g.d == 64 ? forward_d<64>(g, p.splits, q, k, v, o, lse, parts, stream)
                                      : forward_d<128>(g, p.splits, q, k, v, o, lse, parts, stream);
    if (rc != BRA_OK || p.splits == 1) return rc;
    return cross_join(g, p.splits, false, parts, o, lse, stream);
}

bra_status cross_backward_f32(const CrossGeom& g, int splits, const void* q, const void* k, const void* v,
                              const void* o, const float* lse, const void* grad_o, void* dq, void* dk, void* dv,
                              float* delta, float* parts, cudaStream_t stream) {
    const bra_status rc =
        g.d == 32   ? backward_d<32>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, stream)
        : g.d == 64 ? backward_d<64>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, stream)
                    : backward_d<128>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, stream);
    if (rc != BRA_OK || splits == 1) return rc;
    return cross_backward_join(g, splits, false, parts, dk, dv, stream);
}

}  // namespace bra
