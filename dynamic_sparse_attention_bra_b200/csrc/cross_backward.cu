// Gradients of the cross attention, bf16, on warp-level tensor-core products.
// With P = 2^(s' - lse') rebuilt from the forward's log sums,
//   dP = dO V^T,  D_r = <dO_r, O_r>,  dS = P (dP - D),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
// summed over the rows of a state head's group.  Two kernels, neither of
// which adds to memory that another CTA adds to, so results repeat bit for bit:
//   dQ      a CTA owns 64 rows (four warps x 16) and streams the states in
//           tiles of 64; it also forms D and stores it for the second kernel.
//           <dO, O> of the stored bf16 O is only a first value D0: its error
//           2^-9 |dO| |O| multiplies every state alike, so that in dQ it adds up
//           to (D - D0) sum_j P_j k_j, ten times the roundings' share over
//           some thousand states whose K has a mean.  Since sum_j P_j = 1, the
//           row sum of P (dP - D0) is D - D0; with a second accumulator for
//           sum_j P_j k_j the kernel takes the error out at its end.  The sum is
//           that of the rounded dS, so that the roundings' own sum goes with it;
//   dK, dV  a CTA owns 64 states (four warps x 16) and streams the group's
//           rows in tiles of 64, with the transposed scores S^T = K Q^T, so
//           that P^T and dS^T are already the first operands of their products.
// The scores are built twice (8 products in place of 5): the price of sums
// without atomics and of the exact D.  Where the state tiles leave SMs idle the rows are split
// over CTAs and fp32 parts are joined in order.
// Scores, P, dP, D and all sums are fp32; P and dS are rounded once to bf16 as
// operands, gradients once at the end.
#include "cross_tile.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;
using wmma16::mma16816;

constexpr int kThreads = 128;

template <int D>
constexpr uint32_t tile_bytes() { return 64u * D * 2u; }

// Fragments of a 16-row operand: kept in registers where they are few.
template <int D>
struct RowFrags {
    static constexpr bool kKeep = D <= 64;
    uint32_t a[kKeep ? D / 16 : 1][4];
    uint32_t tile;
    int row0, lane;
    __device__ __forceinline__ void init(uint32_t t, int r0, int ln) {
        tile = t;
        row0 = r0;
        lane = ln;
        if constexpr (kKeep)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) frag_a<D>(t, r0, kk, ln, a[kk]);
    }
    __device__ __forceinline__ void get(int kk, uint32_t (&x)[4]) const {
        if constexpr (kKeep) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = a[kk][i];
        } else {
            frag_a<D>(tile, row0, kk, lane, x);
        }
    }
};

// s[i] = (this warp's 16 rows) x (32 rows of ``tile`` from row0)^T.
template <int D>
__device__ __forceinline__ void scores32(const RowFrags<D>& a, uint32_t tile, int row0, int lane, float (&s)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t x[4];
        a.get(kk, x);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint32_t bf[4];
            frag_nt<D>(tile, row0 + i * 8, kk, lane, bf);
            mma16816(s[i], x[0], x[1], x[2], x[3], bf[0], bf[1]);
            mma16816(s[i + 1], x[0], x[1], x[2], x[3], bf[2], bf[3]);
        }
    }
}

// acc += p (16 x 32, rounded to bf16) x (32 rows of ``tile`` from row0).
template <int D>
__device__ __forceinline__ void accumulate32(const float (&p)[4][4], uint32_t tile, int row0, int lane,
                                             float (&acc)[D / 8][4]) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
        uint32_t a[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            a[x] = ptx::pack_bf16x2(p[2 * kt + (x >> 1)][2 * (x & 1)], p[2 * kt + (x >> 1)][2 * (x & 1) + 1]);
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
            uint32_t bf[4];
            frag_nn<D>(tile, row0 + kt * 16, c, lane, bf);
            mma16816(acc[c], a[0], a[1], a[2], a[3], bf[0], bf[1]);
            mma16816(acc[c + 1], a[0], a[1], a[2], a[3], bf[2], bf[3]);
        }
    }
}

// Both at once: acc += p ..., acc2 += p2 ..., the tile's fragments shared.
template <int D>
__device__ __forceinline__ void accumulate32x2(const float (&p)[4][4], const float (&p2)[4][4], uint32_t tile,
                                               int row0, int lane, float (&acc)[D / 8][4], float (&acc2)[D / 8][4]) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
        uint32_t a[4], a2[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            a[x] = ptx::pack_bf16x2(p[2 * kt + (x >> 1)][2 * (x & 1)], p[2 * kt + (x >> 1)][2 * (x & 1) + 1]);
            a2[x] = ptx::pack_bf16x2(p2[2 * kt + (x >> 1)][2 * (x & 1)], p2[2 * kt + (x >> 1)][2 * (x & 1) + 1]);
        }
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
            uint32_t bf[4];
            frag_nn<D>(tile, row0 + kt * 16, c, lane, bf);
            mma16816(acc[c], a[0], a[1], a[2], a[3], bf[0], bf[1]);
            mma16816(acc[c + 1], a[0], a[1], a[2], a[3], bf[2], bf[3]);
            mma16816(acc2[c], a2[0], a2[1], a2[2], a2[3], bf[0], bf[1]);
            mma16816(acc2[c + 1], a2[0], a2[1], a2[2], a2[3], bf[2], bf[3]);
        }
    }
}

template <int D>
__device__ __forceinline__ void zero(float (&acc)[D / 8][4]) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
}

// 64 rows (queries, or dO) of a row tile; rows past the last are zeros.
template <int D>
__device__ __forceinline__ void load_rows(uint32_t dst, const __nv_bfloat16* base, const CrossGeom& g, int b, int j,
                                          int row0, bool dense) {
    constexpr int kChunks = D / 8;
#pragma unroll
    for (int i = 0; i < 64 * kChunks / kThreads; ++i) {
        const int e = i * kThreads + (int)threadIdx.x, r = e / kChunks, c = e % kChunks;
        const bool on = row0 + r < g.rows;
        const size_t off = !on ? 0 : dense ? cross_o_offset(g, b, j, row0 + r) : cross_q_offset(g, b, j, row0 + r);
        ptx::cp_async16_zfill(dst + tile_offset<D>(r, c), base + off + (on ? c * 8 : 0), on ? 16u : 0u);
    }
}

// ------------------------------------------------------------------ dQ and D
// shared memory: Q | dO | ring of 2 x (K | V) | D, log sums [64] | mask bits
template <int D>
constexpr uint32_t dq_smem() { return 6u * tile_bytes<D>() + 512u + 2u * ValidBits::kWords * 4u; }

template <int D>
__global__ void __launch_bounds__(kThreads)
bra_cross_dq_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                    const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ o,
                    const float* lse, const __nv_bfloat16* __restrict__ go,
                    __nv_bfloat16* __restrict__ dq, float* __restrict__ delta, CrossGeom g, int row_tiles) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr uint32_t kTile = tile_bytes<D>();
    const uint32_t sq = ptx::smem_addr(smem), sg = sq + kTile, ring = sg + kTile;
    float* sd = reinterpret_cast<float*>(smem + 6 * kTile);
    float* sl = sd + 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int id = blockIdx.x;
    const int row0 = (id % row_tiles) * 64;
    id /= row_tiles;
    const int j = id % g.kv_heads, b = id / g.kv_heads;

    grid_dependency_wait();
    const int n = cross_len(g, b), tiles = (n + 63) / 64;
    ValidBits bits{reinterpret_cast<uint32_t*>(smem + 6 * kTile + 512),
                   g.kv_mask ? g.kv_mask + (size_t)b * g.Lk : nullptr, n};
    const __nv_bfloat16* kb = k + (size_t)b * g.k_batch + (size_t)j * D;
    const __nv_bfloat16* vb = v + (size_t)b * g.v_batch + (size_t)j * D;
    load_rows<D>(sq, q, g, b, j, row0, false);
    load_rows<D>(sg, go, g, b, j, row0, true);
    auto fetch = [&](int t) {
        if (t < tiles) {
            bits.reach(t, 0, kThreads);
            const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
            const uint32_t st = ring + (uint32_t)(t & 1) * 2u * kTile;
            load_states<D, kThreads>(st, kb, g.k_row, t, w0, w1);
            load_states<D, kThreads>(st + kTile, vb, g.v_row, t, w0, w1);
        }
        ptx::cp_async_commit();
    };
    fetch(0);
    {  // D0 and the log sums: two threads a row
        const int r = threadIdx.x >> 1, half = threadIdx.x & 1;
        float x = 0.f;
        if (row0 + r < g.rows) {
            const size_t off = cross_o_offset(g, b, j, row0 + r) + half * (D / 2);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                float f[8], h[8];
                unpack16(__ldcg(reinterpret_cast<const uint4*>(o + off) + c), f, (const __nv_bfloat16*)nullptr);
                unpack16(__ldcg(reinterpret_cast<const uint4*>(go + off) + c), h, (const __nv_bfloat16*)nullptr);
#pragma unroll
                for (int e = 0; e < 8; ++e) x = fmaf(f[e], h[e], x);
            }
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        if (half == 0) {
            sd[r] = x;
            float ls = -INFINITY;
            if (row0 + r < g.rows) {
                const size_t at = cross_lse_offset(g, b, j, row0 + r);
                ls = __ldcg(lse + at);
            }
            sl[r] = exponent_offset(ls);
        }
    }
    ptx::cp_async_wait_group<0>();
    __syncthreads();
    RowFrags<D> qa, ga;
    qa.init(sq, warp * 16, lane);
    ga.init(sg, warp * 16, lane);
    const float dr[2] = {sd[warp * 16 + (lane >> 2)], sd[warp * 16 + 8 + (lane >> 2)]};
    const float lr[2] = {sl[warp * 16 + (lane >> 2)], sl[warp * 16 + 8 + (lane >> 2)]};
    const float c2 = g.scale * kLog2e;
    float acc[D / 8][4], mean[D / 8][4], rest[2] = {0.f, 0.f};
    zero<D>(acc);
    zero<D>(mean);
    for (int t = 0; t < tiles; ++t) {
        if (t > 0) {
            ptx::cp_async_wait_group<0>();
            __syncthreads();
        }
        fetch(t + 1);
        const uint32_t st = ring + (uint32_t)(t & 1) * 2u * kTile;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const uint32_t w = bits.word(t, hf);
            if (w == 0u) continue;
            float s[4][4], dp[4][4];
            scores32<D>(qa, st, hf * 32, lane, s);
            scores32<D>(ga, st + kTile, hf * 32, lane, dp);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool on = (w >> (i * 8 + (lane & 3) * 2 + (e & 1))) & 1u;
                    const float p = on ? ptx::ex2(fmaf(s[i][e], c2, -lr[e >> 1])) : 0.f;
                    s[i][e] = __bfloat162float(__float2bfloat16_rn(p * (dp[i][e] - dr[e >> 1])));
                    dp[i][e] = p;
                    rest[e >> 1] += s[i][e];
                }
            accumulate32x2<D>(s, dp, st, hf * 32, lane, acc, mean);
        }
    }
    allow_dependents();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        rest[h] += __shfl_xor_sync(0xffffffffu, rest[h], 1);
        rest[h] += __shfl_xor_sync(0xffffffffu, rest[h], 2);
        const int r = row0 + warp * 16 + h * 8 + (lane >> 2);
        if (r >= g.rows) continue;
        if ((lane & 3) == 0) delta[cross_lse_offset(g, b, j, r)] = dr[h] + rest[h];
        __nv_bfloat16* row = dq + cross_o_offset(g, b, j, r) + (lane & 3) * 2;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t*>(row + i * 8) =
                ptx::pack_bf16x2(fmaf(-rest[h], mean[i][2 * h], acc[i][2 * h]) * g.scale,
                                 fmaf(-rest[h], mean[i][2 * h + 1], acc[i][2 * h + 1]) * g.scale);
    }
}

// -------------------------------------------------------------------- dK, dV
// shared memory: K | V | ring of 2 x (Q | dO) | 2 x (log sums, D) [64]
template <int D>
constexpr uint32_t dkv_smem() { return 6u * tile_bytes<D>() + 1024u; }

template <int D>
__global__ void __launch_bounds__(kThreads)
bra_cross_dkv_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                     const __nv_bfloat16* __restrict__ v, const float* lse,
                     const __nv_bfloat16* __restrict__ go, const float* delta,
                     __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, float* __restrict__ parts,
                     CrossGeom g, int key_tiles, int splits) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr uint32_t kTile = tile_bytes<D>();
    const uint32_t sk = ptx::smem_addr(smem), sv = sk + kTile, ring = sv + kTile, stats = ring + 4 * kTile;
    const float* stat = reinterpret_cast<const float*>(smem + 6 * kTile);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    const int t0 = split * per, t1 = (w[0] | w[1]) ? min(all, t0 + per) : t0;  // masked states: zeros
    load_states<D, kThreads>(sk, k + (size_t)b * g.k_batch + (size_t)j * D, g.k_row, kt, w[0], w[1]);
    load_states<D, kThreads>(sv, v + (size_t)b * g.v_batch + (size_t)j * D, g.v_row, kt, w[0], w[1]);
    auto fetch = [&](int t) {
        if (t < t1) {
            const uint32_t st = ring + (uint32_t)((t - t0) & 1) * 2u * kTile;
            load_rows<D>(st, q, g, b, j, t * 64, false);
            load_rows<D>(st + kTile, go, g, b, j, t * 64, true);
            // thread = one row's log sum (first 64) or D (last 64)
            const int r = threadIdx.x & 63;
            const bool on = t * 64 + r < g.rows;
            const float* src = threadIdx.x < 64 ? lse : delta;
            ptx::cp_async4(stats + (uint32_t)((t - t0) & 1) * 512u + threadIdx.x * 4u,
                           src + (on ? cross_lse_offset(g, b, j, t * 64 + r) : 0), on ? 4u : 0u);
        }
        ptx::cp_async_commit();
    };
    fetch(t0);
    ptx::cp_async_wait_group<0>();
    __syncthreads();
    RowFrags<D> ka, va;
    ka.init(sk, warp * 16, lane);
    va.init(sv, warp * 16, lane);
    bool on[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = warp * 16 + h * 8 + (lane >> 2);
        on[h] = ((r < 32 ? w[0] : w[1]) >> (r & 31)) & 1u;
    }
    const float c2 = g.scale * kLog2e;
    float ak[D / 8][4], av[D / 8][4];
    zero<D>(ak);
    zero<D>(av);
    for (int t = t0; t < t1; ++t) {
        if (t > t0) {
            ptx::cp_async_wait_group<0>();
            __syncthreads();
        }
        fetch(t + 1);
        const uint32_t st = ring + (uint32_t)((t - t0) & 1) * 2u * kTile;
        const float* sl = stat + ((t - t0) & 1) * 128;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float s[4][4], dp[4][4];
            scores32<D>(ka, st, hf * 32, lane, s);
            scores32<D>(va, st + kTile, hf * 32, lane, dp);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int col = hf * 32 + i * 8 + (lane & 3) * 2 + x;
                    const float off = exponent_offset(sl[col]), dd = sl[64 + col];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p = on[h] ? ptx::ex2(fmaf(s[i][2 * h + x], c2, -off)) : 0.f;
                        s[i][2 * h + x] = p;
                        dp[i][2 * h + x] = p * (dp[i][2 * h + x] - dd);
                    }
                }
            accumulate32<D>(s, st + kTile, hf * 32, lane, av);
            accumulate32<D>(dp, st, hf * 32, lane, ak);
        }
    }
    ptx::cp_async_wait_all();
    allow_dependents();
    const size_t elems = (size_t)g.B * g.Lk * g.kv_heads * D;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int key = kt * 64 + warp * 16 + h * 8 + (lane >> 2);
        if (key >= g.Lk) continue;
        if (!on[h]) {  // an infinite gradient times its P of zero has made these sums NaN
#pragma unroll
            for (int i = 0; i < D / 8; ++i) ak[i][2 * h] = ak[i][2 * h + 1] = av[i][2 * h] = av[i][2 * h + 1] = 0.f;
        }
        const size_t at = (((size_t)b * g.Lk + key) * g.kv_heads + j) * D + (lane & 3) * 2;
        if (splits > 1) {
            float* pk = parts + (size_t)split * 2 * elems + at;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                *reinterpret_cast<float2*>(pk + i * 8) = make_float2(ak[i][2 * h] * g.scale, ak[i][2 * h + 1] * g.scale);
                *reinterpret_cast<float2*>(pk + elems + i * 8) = make_float2(av[i][2 * h], av[i][2 * h + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                *reinterpret_cast<uint32_t*>(dk + at + i * 8) =
                    ptx::pack_bf16x2(ak[i][2 * h] * g.scale, ak[i][2 * h + 1] * g.scale);
                *reinterpret_cast<uint32_t*>(dv + at + i * 8) = ptx::pack_bf16x2(av[i][2 * h], av[i][2 * h + 1]);
            }
        }
    }
}

// Sums the row splits' parts in order; thread = four elements of dK, then dV.
template <typename T>
__global__ void __launch_bounds__(256)
bra_cross_dkv_join_kernel(const float* parts, T* __restrict__ dk, T* __restrict__ dv, size_t elems,
                          int splits) {
    grid_dependency_wait();
    allow_dependents();
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= 2 * elems) return;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < splits; ++s) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(parts + (size_t)s * 2 * elems + i));
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
    }
    T* out = i < elems ? dk + i : dv + (i - elems);  // elems is a multiple of 4
    out[0] = from_f32<T>(x.x);
    out[1] = from_f32<T>(x.y);
    out[2] = from_f32<T>(x.z);
    out[3] = from_f32<T>(x.w);
}

template <int D>
bra_status launch_d(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, const void* o,
                    const float* lse, const void* go, void* dq, void* dk, void* dv, float* delta, float* parts,
                    cudaStream_t stream) {
    using T = __nv_bfloat16;
    if (!allow_shared<bra_cross_dq_kernel<D>>(dq_smem<D>()) || !allow_shared<bra_cross_dkv_kernel<D>>(dkv_smem<D>()))
        return BRA_ERR_CUDA;
    const int row_tiles = (g.rows + 63) / 64, key_tiles = (g.Lk + 63) / 64;
    const long long grid_q = (long long)row_tiles * g.kv_heads * g.B;
    const long long grid_k = (long long)key_tiles * splits * g.kv_heads * g.B;
    if (grid_q > 0x7fffffffLL || grid_k > 0x7fffffffLL) return BRA_ERR_UNSUPPORTED;
    cudaError_t e = launch_after_previous(bra_cross_dq_kernel<D>, dim3((unsigned)grid_q), dim3(kThreads), dq_smem<D>(),
                                          stream, (const T*)q, (const T*)k, (const T*)v, (const T*)o, lse,
                                          (const T*)go, (T*)dq, delta, g, row_tiles);
    if (e != cudaSuccess) return BRA_ERR_CUDA;
    if (grid_k == 0) return BRA_OK;
    e = launch_after_previous(bra_cross_dkv_kernel<D>, dim3((unsigned)grid_k), dim3(kThreads), dkv_smem<D>(), stream,
                              (const T*)q, (const T*)k, (const T*)v, lse, (const T*)go, (const float*)delta, (T*)dk,
                              (T*)dv, parts, g, key_tiles, splits);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace

// Enough row splits for two CTAs on each SM (fp32: three at d = 32, one CTA
// of twice the warps otherwise), each of at least four row tiles.
int cross_backward_splits(const CrossGeom& g, bool bf16) {
    if (bf16 && cross_tc_backward_covers(g)) return cross_tc_backward_splits(g);
    const int slots = sm_count() * (bf16 ? 2 : g.d == 32 ? 3 : 1);
    const long long ctas = (long long)((g.Lk + 63) / 64) * g.kv_heads * g.B;
    if (slots <= 0 || ctas <= 0 || ctas >= slots) return 1;
    long long s = slots / ctas;
    const long long most = ((g.rows + 63) / 64) / 4;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

bra_status cross_backward_bf16(const CrossGeom& g, int splits, const void* q, const void* k, const void* v,
                               const void* o, const float* lse, const void* grad_o, void* dq, void* dk, void* dv,
                               float* delta, float* parts, int* status, cudaStream_t stream) {
    const bra_status rc =
        cross_tc_backward_covers(g)
            ? cross_backward_tc(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, status, stream)
        : g.d == 32 ? launch_d<32>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, stream)
        : g.d == 64 ? launch_d<64>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, stream)
                    : launch_d<128>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, stream);
    if (rc != BRA_OK || splits == 1) return rc;
    return cross_backward_join(g, splits, true, parts, dk, dv, stream);
}

bra_status cross_backward_join(const CrossGeom& g, int splits, bool bf16, const float* parts, void* dk, void* dv,
                               cudaStream_t stream) {
    const size_t elems = (size_t)g.B * g.Lk * g.kv_heads * g.d;
    const size_t grid = (2 * elems / 4 + 255) / 256;
    if (grid == 0) return BRA_OK;
    if (grid > 0x7fffffffu) return BRA_ERR_UNSUPPORTED;
    const cudaError_t e =
        bf16 ? launch_after_previous(bra_cross_dkv_join_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(256), 0,
                                     stream, parts, static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv),
                                     elems, splits)
             : launch_after_previous(bra_cross_dkv_join_kernel<float>, dim3((unsigned)grid), dim3(256), 0, stream,
                                     parts, static_cast<float*>(dk), static_cast<float*>(dv), elems, splits);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace bra
