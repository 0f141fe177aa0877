// Cross attention and its gradients in fp32 on tensor cores (the formulas are
// those of the bf16 kernels).  Every fp32 factor x is split (as by Dekker, "A floating-
// point technique for extending the available precision", 1971) into x rounded to tf32
// and the rest, x - that, which is exact; a product of two factors is then three tf32 products,
//   x y = xh yh + xh yl + xl yh  (+ xl yl, below 2^-20 of x y),
// summed in fp32: some 2^-21 of relative error a factor, the order of fp32's own
// roundings in a sum.  Three products cost 24 clocks of a warp's tensor unit for
// 1024 multiply-adds, CUDA cores 32 and more for their shared-memory reads: 8 x
// 784 rows over 333 states, 4 heads of 32, take 32 us, a form on CUDA cores 42 us.
//
// Fragments of m16n8k8 are read as 16-byte words: the inner index of the scores
// takes a thread's four channels 4 t .. 4 t + 3 for two steps, that of the sums
// the states 2 t, 2 t + 1 that the thread already has P of, and their columns the
// channels 4 g .. 4 g + 3 of four n8 tiles; rows of a tile are swizzled so that
// both kinds of reads fall in distinct banks.
#include "cross_tile.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;

// ---------------------------------------------------------------- fragments

__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;  // (integer operations: conversions run at a quarter of their rate)
    lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A 16 x 8 operand in its two parts.
struct Split {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ void set(float a0, float a1, float a2, float a3) {
        split(a0, hi[0], lo[0]);
        split(a1, hi[1], lo[1]);
        split(a2, hi[2], lo[2]);
        split(a3, hi[3], lo[3]);
    }
    // d += the first parts' product, r += the two others
    __device__ __forceinline__ void times(float (&d)[4], float (&r)[4], float b0, float b1) const {
        uint32_t h0, l0, h1, l1;
        split(b0, h0, l0);
        split(b1, h1, l1);
        mma_tf32(r, lo, h0, h1);
        mma_tf32(r, hi, l0, l1);
        mma_tf32(d, hi, h0, h1);
    }
};

// Byte offset of 16-byte chunk c of row r.
template <int D>
__device__ __forceinline__ uint32_t f32_offset(int r, int c) {
    return (uint32_t)(r * D * 4 + ((c ^ ((((r >> 1) & 3) << 1) ^ ((r & 1) << 2))) << 4));
}
__device__ __forceinline__ float4 lds128(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    return v;
}

// s[i] = (16 rows of tile ``a`` from a0) x (rows b0 + 8 i .. of tile ``b``)^T
template <int D, int N>
__device__ __forceinline__ void scores(uint32_t a, int a0, uint32_t b, int b0, int lane, float (&s)[N][4]) {
    const int gq = lane >> 2, t4 = lane & 3;
    float r[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = r[i][e] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        const float4 x = lds128(a + f32_offset<D>(a0 + gq, c * 4 + t4)), y = lds128(a + f32_offset<D>(a0 + 8 + gq, c * 4 + t4));
        Split f[2];
        f[0].set(x.x, y.x, x.y, y.y);
        f[1].set(x.z, y.z, x.w, y.w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float4 z = lds128(b + f32_offset<D>(b0 + 8 * i + gq, c * 4 + t4));
            f[0].times(s[i], r[i], z.x, z.y);
            f[1].times(s[i], r[i], z.z, z.w);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] += r[i][e];
}

// acc += p (16 rows x 8 N columns, as scores leaves them) x (8 N rows of ``tile`` from row0),
// for the MC blocks of 32 channels from m0: acc[4 m + x] has the channels
// 32 (m0 + m) + 8 t + x (first of each pair) and + 4 (second).
// The tensor unit cuts off what falls below its sum, always towards zero: over some
// hundred products into one sum that is a bias of 2^-18.  So a tile's products make
// sums of their own, of N products the first parts' and of 2 N the small others',
// which are added to acc in fp32, rounded to nearest.
template <int D, int N, int MC>
__device__ __forceinline__ void accumulate(const float (&p)[N][4], uint32_t tile, int row0, int m0, int lane,
                                           float (&acc)[4 * MC][4]) {
    const int gq = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int m = 0; m < MC; ++m) {
        float sum[4][4], low[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[x][e] = low[x][e] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            Split f;
            f.set(p[i][0], p[i][2], p[i][1], p[i][3]);
            const int r = row0 + 8 * i + 2 * t4, c = (m0 + m) * 8 + gq;
            const float4 x = lds128(tile + f32_offset<D>(r, c)), y = lds128(tile + f32_offset<D>(r + 1, c));
            f.times(sum[0], low[0], x.x, y.x);
            f.times(sum[1], low[1], x.y, y.y);
            f.times(sum[2], low[2], x.z, y.z);
            f.times(sum[3], low[3], x.w, y.w);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[4 * m + x][e] += sum[x][e] + low[x][e];
    }
}

// The same with the factors' first parts alone (2^-10), for what need not be exact.
template <int D, int N, int MC>
__device__ __forceinline__ void accumulate_coarse(const float (&p)[N][4], uint32_t tile, int row0, int m0, int lane,
                                                  float (&acc)[4 * MC][4]) {
    const int gq = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t a[4] = {__float_as_uint(p[i][0]), __float_as_uint(p[i][2]), __float_as_uint(p[i][1]),
                               __float_as_uint(p[i][3])};
        const int r = row0 + 8 * i + 2 * t4;
#pragma unroll
        for (int m = 0; m < MC; ++m) {
            const int c = (m0 + m) * 8 + gq;
            const float4 x = lds128(tile + f32_offset<D>(r, c)), y = lds128(tile + f32_offset<D>(r + 1, c));
            mma_tf32(acc[4 * m], a, __float_as_uint(x.x), __float_as_uint(y.x));
            mma_tf32(acc[4 * m + 1], a, __float_as_uint(x.y), __float_as_uint(y.y));
            mma_tf32(acc[4 * m + 2], a, __float_as_uint(x.z), __float_as_uint(y.z));
            mma_tf32(acc[4 * m + 3], a, __float_as_uint(x.w), __float_as_uint(y.w));
        }
    }
}

template <int N>
__device__ __forceinline__ void zero(float (&acc)[N][4]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
}

// Row h (0: gq, 1: gq + 8) of acc, times f, to its channels of ``row``: 32 bytes of every 32 channels a thread.
template <int N>
__device__ __forceinline__ void store_row(float* row, const float (&acc)[N][4], int h, float f, int t4) {
#pragma unroll
    for (int m = 0; m < N / 4; ++m) {
        float4* dst = reinterpret_cast<float4*>(row + 32 * m + 8 * t4);
        dst[0] = make_float4(acc[4 * m][2 * h] * f, acc[4 * m + 1][2 * h] * f, acc[4 * m + 2][2 * h] * f,
                             acc[4 * m + 3][2 * h] * f);
        dst[1] = make_float4(acc[4 * m][2 * h + 1] * f, acc[4 * m + 1][2 * h + 1] * f, acc[4 * m + 2][2 * h + 1] * f,
                             acc[4 * m + 3][2 * h + 1] * f);
    }
}

// -------------------------------------------------------------------- loads

template <int D, int THREADS>
__device__ __forceinline__ void load_states_f32(uint32_t dst, const float* base, long long step, int t, uint32_t w0,
                                                uint32_t w1) {
    constexpr int kChunks = D / 4;
#pragma unroll 8
    for (int i = 0; i < 64 * kChunks / THREADS; ++i) {
        const int e = i * THREADS + (int)threadIdx.x, r = e / kChunks, c = e % kChunks;
        const bool on = ((r < 32 ? w0 : w1) >> (r & 31)) & 1u;
        ptx::cp_async16_zfill(dst + f32_offset<D>(r, c), on ? base + (size_t)(t * 64 + r) * step + c * 4 : base,
                              on ? 16u : 0u);
    }
}

template <int D, int THREADS, int ROWS>
__device__ __forceinline__ void load_rows_f32(uint32_t dst, const float* base, const CrossGeom& g, int b, int j,
                                              int row0, bool dense) {
    constexpr int kChunks = D / 4;
    for (int e = threadIdx.x; e < ROWS * kChunks; e += THREADS) {
        const int r = e / kChunks, c = e % kChunks;
        const bool on = row0 + r < g.rows;
        const size_t off = !on ? 0 : dense ? cross_o_offset(g, b, j, row0 + r) : cross_q_offset(g, b, j, row0 + r);
        ptx::cp_async16_zfill(dst + f32_offset<D>(r, c), base + off + (on ? c * 4 : 0), on ? 16u : 0u);
    }
}

template <int D>
constexpr uint32_t tile_bytes() { return 64u * D * 4u; }

// ------------------------------------------------------------------- forward
// WM warps share the rows (16 each), WN the 64 states of a tile, as in cross_mma.cu.
// shared memory: Q | ring of 2 x (K | V) (join of the WN parts) | mask bits
template <int D, int WM, int WN>
struct Fwd {
    static constexpr int kRows = 16 * WM, kThreads = 32 * WM * WN;
    static constexpr uint32_t kQ = (uint32_t)kRows * D * 4u, kRing = 4u * tile_bytes<D>();
    static constexpr uint32_t kJoin = WN > 1 ? (uint32_t)WN * kRows * (D + 2) * 4u : 0u;
    static constexpr uint32_t kBytes = kQ + (kRing > kJoin ? kRing : kJoin) + 2u * ValidBits::kWords * 4u;
};

template <int D, int WM, int WN>
__global__ void __launch_bounds__(32 * WM * WN)
bra_cross_tf32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                      float* __restrict__ o, float* __restrict__ lse, CrossParts parts, CrossGeom g, int row_tiles,
                      int splits) {
    using S = Fwd<D, WM, WN>;
    constexpr int kThreads = S::kThreads, KW = 64 / WN, N = KW / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sq = ptx::smem_addr(smem), ring = sq + S::kQ;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t4 = lane & 3;
    const int wm = warp % WM, wn = warp / WM;
    int id = blockIdx.x;
    const int row0 = (id % row_tiles) * S::kRows;
    id /= row_tiles;
    const int split = id % splits;
    id /= splits;
    const int j = id % g.kv_heads, b = id / g.kv_heads;
    grid_dependency_wait();
    const int n = cross_len(g, b), all = (n + 63) / 64, per = (all + splits - 1) / splits;
    const int t0 = split * per, t1 = min(all, t0 + per);
    ValidBits bits{reinterpret_cast<uint32_t*>(smem + S::kBytes - 2u * ValidBits::kWords * 4u),
                   g.kv_mask ? g.kv_mask + (size_t)b * g.Lk : nullptr, n};
    load_rows_f32<D, kThreads, S::kRows>(sq, q, g, b, j, row0, false);
    auto fetch = [&](int t) {
        if (t < t1) {
            bits.reach(t, t0, kThreads);
            const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
            const uint32_t st = ring + (uint32_t)((t - t0) & 1) * 2u * tile_bytes<D>();
            load_states_f32<D, kThreads>(st, k + (size_t)b * g.k_batch + (size_t)j * D, g.k_row, t, w0, w1);
            load_states_f32<D, kThreads>(st + tile_bytes<D>(), v + (size_t)b * g.v_batch + (size_t)j * D, g.v_row, t, w0,
                                         w1);
        }
        ptx::cp_async_commit();
    };
    fetch(t0);
    const float sl = g.scale * kLog2e;
    float acc[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    zero(acc);
    for (int t = t0; t < t1; ++t) {
        ptx::cp_async_wait_group<0>();
        __syncthreads();  // this tile has landed, and everyone is done with the last
        fetch(t + 1);
        const uint32_t st = ring + (uint32_t)((t - t0) & 1) * 2u * tile_bytes<D>();
        const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
        if ((w0 | w1) == 0u) continue;
        float s[N][4];
        scores<D, N>(sq, wm * 16, st, wn * KW, lane, s);
        if ((w0 & w1) != 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = wn * KW + i * 8 + t4 * 2;
                const uint32_t w = (c < 32 ? w0 : w1) >> (c & 31);
                if (!(w & 1u)) s[i][0] = s[i][2] = -INFINITY;
                if (!(w & 2u)) s[i][1] = s[i][3] = -INFINITY;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i) mx = ptx::max3(mx, s[i][2 * h], s[i][2 * h + 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[h], mx * sl), mu = mn == -INFINITY ? 0.f : mn;
            const float alpha = ptx::ex2(m[h] - mu);
            m[h] = mn;
            l[h] *= alpha;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 2 * h; e < 2 * h + 2; ++e) {
                    s[i][e] = ptx::ex2(fmaf(s[i][e], sl, -mu));
                    l[h] += s[i][e];
                }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                acc[i][2 * h] *= alpha;
                acc[i][2 * h + 1] *= alpha;
            }
        }
        accumulate<D, N, D / 32>(s, st + tile_bytes<D>(), wn * KW, 0, lane, acc);
    }
    ptx::cp_async_wait_all();
    allow_dependents();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if constexpr (WN > 1) {
        float* jo = reinterpret_cast<float*>(smem + S::kQ);  // [WN][rows][D]
        float* jm = jo + WN * S::kRows * D;                  // [WN][rows][2]
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = wn * S::kRows + wm * 16 + h * 8 + gq;
            store_row(jo + (size_t)r * D, acc, h, 1.f, t4);
            if (t4 == 0) {
                jm[r * 2] = m[h];
                jm[r * 2 + 1] = l[h];
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < S::kRows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            if (row0 + r >= g.rows) continue;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int w = 0; w < WN; ++w) mm = fmaxf(mm, jm[(w * S::kRows + r) * 2]);
            const float mu = mm == -INFINITY ? 0.f : mm;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                const float f = ptx::ex2(jm[(w * S::kRows + r) * 2] - mu);
                const float4 y = *reinterpret_cast<const float4*>(jo + (size_t)(w * S::kRows + r) * D + c);
                ll = fmaf(jm[(w * S::kRows + r) * 2 + 1], f, ll);
                x.x = fmaf(y.x, f, x.x);
                x.y = fmaf(y.y, f, x.y);
                x.z = fmaf(y.z, f, x.z);
                x.w = fmaf(y.w, f, x.w);
            }
            if (splits > 1) {
                const size_t at = ((size_t)(split * g.B + b) * g.kv_heads + j) * g.rows + row0 + r;
                *reinterpret_cast<float4*>(parts.o + at * D + c) = x;
                if (c == 0) parts.ml[at] = make_float2(mm, ll);
            } else {
                const float inv = inverse_sum(ll);
                *reinterpret_cast<float4*>(o + cross_o_offset(g, b, j, row0 + r) + c) =
                    make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
                if (c == 0 && lse)
                    lse[cross_lse_offset(g, b, j, row0 + r)] = log_sum(mm, ll);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = row0 + wm * 16 + h * 8 + gq;
            if (r >= g.rows) continue;
            if (splits > 1) {
                const size_t at = ((size_t)(split * g.B + b) * g.kv_heads + j) * g.rows + r;
                store_row(parts.o + at * D, acc, h, 1.f, t4);
                if (t4 == 0) parts.ml[at] = make_float2(m[h], l[h]);
            } else {
                store_row(o + cross_o_offset(g, b, j, r), acc, h, inverse_sum(l[h]), t4);
                if (t4 == 0 && lse)
                    lse[cross_lse_offset(g, b, j, r)] = log_sum(m[h], l[h]);
            }
        }
    }
}

// ----------------------------------------------------------------- gradients
// Eight warps: 16 rows of a tile of 64 each pair, and of a pair each warp the scores
// of 32 columns.  d = 32: it also sums over these, and the pair joins its sums at the
// end.  d = 64, 128: registers do not hold the sums of all channels, so the pair
// exchanges P and dS through shared memory, in fragment order, and each warp sums half
// of the channels over all 64 columns.
constexpr int kThreads = 256;

template <int D>
struct Grad {
    static constexpr bool kExchange = D > 32;
    static constexpr int kBlocks = kExchange ? D / 64 : 1;  // of 32 channels that a warp sums
    static constexpr uint32_t kShare = 4u * 8u * 32u * 16u;  // one exchanged matrix (or the join's sums)
    // four tiles, or the rows' two and a ring of two stages of two | exchange | statistics | mask bits
    static constexpr uint32_t kOffShare = 6u * tile_bytes<D>();
    static constexpr uint32_t kOffStat = kOffShare + 2u * kShare;
    static constexpr uint32_t kBytes = kOffStat + 1024u + 2u * ValidBits::kWords * 4u;
    static_assert(kBytes <= 227u * 1024u, "shared memory");
};

// This warp's 16 x 32 part of a matrix to, or the pair's 16 x 64 from, shared memory.
__device__ __forceinline__ void give(uint32_t share, int pair, int half, int lane, const float (&s)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ptx::st_shared_v4(share + (uint32_t)(((pair * 8 + half * 4 + i) * 32 + lane) * 16), __float_as_uint(s[i][0]),
                          __float_as_uint(s[i][1]), __float_as_uint(s[i][2]), __float_as_uint(s[i][3]));
}
__device__ __forceinline__ void take(uint32_t share, int pair, int lane, float (&s)[8][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 v = lds128(share + (uint32_t)(((pair * 8 + i) * 32 + lane) * 16));
        s[i][0] = v.x;
        s[i][1] = v.y;
        s[i][2] = v.z;
        s[i][3] = v.w;
    }
}
// d = 32: the right warp's sums (4 x 4 a thread) added to the left's; the whole CTA calls it.
__device__ __forceinline__ void join_pair(uint32_t share, int pair, int half, int lane, float (&acc)[4][4]) {
    if (half == 1) give(share, pair, 0, lane, acc);
    __syncthreads();
    if (half == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = lds128(share + (uint32_t)(((pair * 8 + i) * 32 + lane) * 16));
            acc[i][0] += v.x;
            acc[i][1] += v.y;
            acc[i][2] += v.z;
            acc[i][3] += v.w;
        }
    }
}

// dQ and D.  <dO, O> is D0; what it lacks to D multiplies sum_j P_j k_j in dQ and is
// taken out at the end, as in the bf16 kernel: O's 2^-20 would make 10^-5 of dQ over
// 8000 states.  That sum needs no second parts.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 32 ? 2 : 1)
bra_cross_tf32_dq_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                         const float* __restrict__ o, const float* lse, const float* __restrict__ go,
                         float* __restrict__ dq, float* delta, CrossGeom g, int row_tiles) {
    using G = Grad<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr uint32_t kTile = tile_bytes<D>();
    const uint32_t sq = ptx::smem_addr(smem), sg = sq + kTile, ring = sg + kTile, share = sq + G::kOffShare;
    float* sd = reinterpret_cast<float*>(smem + G::kOffStat);  // D0, -, log sums; at the end a row's two sums of dS
    float* sl = sd + 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t4 = lane & 3;
    const int pair = warp & 3, half = warp >> 2;
    int id = blockIdx.x;
    const int row0 = (id % row_tiles) * 64;
    id /= row_tiles;
    const int j = id % g.kv_heads, b = id / g.kv_heads;
    grid_dependency_wait();
    const int n = cross_len(g, b), tiles = (n + 63) / 64;
    ValidBits bits{reinterpret_cast<uint32_t*>(smem + G::kOffStat + 1024u),
                   g.kv_mask ? g.kv_mask + (size_t)b * g.Lk : nullptr, n};
    load_rows_f32<D, kThreads, 64>(sq, q, g, b, j, row0, false);
    load_rows_f32<D, kThreads, 64>(sg, go, g, b, j, row0, true);
    auto fetch = [&](int t) {
        if (t < tiles) {
            bits.reach(t, 0, kThreads);
            const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
            const uint32_t st = ring + (uint32_t)(t & 1) * 2u * kTile;
            load_states_f32<D, kThreads>(st, k + (size_t)b * g.k_batch + (size_t)j * D, g.k_row, t, w0, w1);
            load_states_f32<D, kThreads>(st + kTile, v + (size_t)b * g.v_batch + (size_t)j * D, g.v_row, t, w0, w1);
        }
        ptx::cp_async_commit();
    };
    fetch(0);
    {  // D0 and the log sums: four threads a row
        const int r = threadIdx.x >> 2, part = threadIdx.x & 3;
        float x = 0.f;
        if (row0 + r < g.rows) {
            const size_t off = cross_o_offset(g, b, j, row0 + r) + part * (D / 4);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(o + off) + c);
                const float4 h = __ldcg(reinterpret_cast<const float4*>(go + off) + c);
                x = fmaf(f.x, h.x, x);
                x = fmaf(f.y, h.y, x);
                x = fmaf(f.z, h.z, x);
                x = fmaf(f.w, h.w, x);
            }
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (part == 0) {
            sd[r] = x;
            sl[r] = exponent_offset(row0 + r < g.rows ? __ldcg(lse + cross_lse_offset(g, b, j, row0 + r)) : -INFINITY);
        }
    }
    const float c2 = g.scale * kLog2e;
    float acc[4 * G::kBlocks][4], mean[4 * G::kBlocks][4], rest[2] = {0.f, 0.f};
    zero(acc);
    zero(mean);
    for (int t = 0; t < tiles; ++t) {
        ptx::cp_async_wait_group<0>();
        __syncthreads();
        fetch(t + 1);
        const uint32_t st = ring + (uint32_t)(t & 1) * 2u * kTile;
        const uint32_t w = bits.word(t, half);
        if (!G::kExchange && w == 0u) continue;
        float s[4][4], dp[4][4];
        scores<D, 4>(sq, pair * 16, st, half * 32, lane, s);
        scores<D, 4>(sg, pair * 16, st + kTile, half * 32, lane, dp);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = pair * 16 + (e >> 1) * 8 + gq;
            const float off = sl[r], dd = sd[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool on = (w >> (i * 8 + t4 * 2 + (e & 1))) & 1u;
                const float p = on ? ptx::ex2(fmaf(s[i][e], c2, -off)) : 0.f;
                s[i][e] = on ? p * (dp[i][e] - dd) : 0.f;  // (an infinite dO makes NaN of dP)
                dp[i][e] = p;
                rest[e >> 1] += s[i][e];
            }
        }
        if constexpr (G::kExchange) {
            give(share, pair, half, lane, s);
            give(share + G::kShare, pair, half, lane, dp);
            __syncthreads();
            float x[8][4];
            take(share, pair, lane, x);
            accumulate<D, 8, G::kBlocks>(x, st, 0, half * G::kBlocks, lane, acc);
            take(share + G::kShare, pair, lane, x);
            accumulate_coarse<D, 8, G::kBlocks>(x, st, 0, half * G::kBlocks, lane, mean);
        } else {
            accumulate<D, 4, 1>(s, st, half * 32, 0, lane, acc);
            accumulate_coarse<D, 4, 1>(dp, st, half * 32, 0, lane, mean);
        }
    }
    ptx::cp_async_wait_all();
    allow_dependents();
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the row's sum of dS over both warps' columns
        rest[h] += __shfl_xor_sync(0xffffffffu, rest[h], 1);
        rest[h] += __shfl_xor_sync(0xffffffffu, rest[h], 2);
        if (t4 == 0) sl[64 + half * 64 + pair * 16 + h * 8 + gq] = rest[h];
    }
    __syncthreads();
    if constexpr (!G::kExchange) {
        join_pair(share, pair, half, lane, acc);
        join_pair(share + G::kShare, pair, half, lane, mean);
        if (half == 1) return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int y = pair * 16 + h * 8 + gq, r = row0 + y;
        const float left = sl[64 + y] + sl[128 + y];
#pragma unroll
        for (int i = 0; i < 4 * G::kBlocks; ++i)
#pragma unroll
            for (int e = 2 * h; e < 2 * h + 2; ++e) acc[i][e] = fmaf(-left, mean[i][e], acc[i][e]);
        if (r >= g.rows) continue;
        store_row(dq + cross_o_offset(g, b, j, r) + half * G::kBlocks * 32, acc, h, g.scale, t4);
        if (t4 == 0 && half == 0) delta[cross_lse_offset(g, b, j, r)] = sd[y] + left;
    }
}

// dK, dV: the rows are 64 states, the columns the group's rows of queries.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 32 ? 2 : 1)
bra_cross_tf32_dkv_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                          const float* lse, const float* __restrict__ go, const float* delta, float* __restrict__ dk,
                          float* __restrict__ dv, float* parts, CrossGeom g, int key_tiles, int splits) {
    using G = Grad<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr uint32_t kTile = tile_bytes<D>();
    const uint32_t sk = ptx::smem_addr(smem), sv = sk + kTile, ring = sv + kTile, share = sk + G::kOffShare;
    float* stat = reinterpret_cast<float*>(smem + G::kOffStat);  // [stage] (log sums, D) [64]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t4 = lane & 3;
    const int pair = warp & 3, half = warp >> 2;
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
    load_states_f32<D, kThreads>(sk, k + (size_t)b * g.k_batch + (size_t)j * D, g.k_row, kt, w[0], w[1]);
    load_states_f32<D, kThreads>(sv, v + (size_t)b * g.v_batch + (size_t)j * D, g.v_row, kt, w[0], w[1]);
    auto fetch = [&](int t) {
        if (t < t1) {
            const int x = (t - t0) & 1;
            const uint32_t st = ring + (uint32_t)x * 2u * kTile;
            load_rows_f32<D, kThreads, 64>(st, q, g, b, j, t * 64, false);
            load_rows_f32<D, kThreads, 64>(st + kTile, go, g, b, j, t * 64, true);
            if (threadIdx.x < 128) {  // a row's log sum (first 64 threads) or D
                const int r = threadIdx.x & 63;
                const bool in = t * 64 + r < g.rows;
                const float* src = threadIdx.x < 64 ? lse : delta;
                ptx::cp_async4(ptx::smem_addr(stat) + (uint32_t)(x * 128 + (int)threadIdx.x) * 4u,
                               src + (in ? cross_lse_offset(g, b, j, t * 64 + r) : 0), in ? 4u : 0u);
            }
        }
        ptx::cp_async_commit();
    };
    fetch(t0);
    bool on[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = pair * 16 + h * 8 + gq;
        on[h] = ((r < 32 ? w[0] : w[1]) >> (r & 31)) & 1u;
    }
    const float c2 = g.scale * kLog2e;
    float ak[4 * G::kBlocks][4], av[4 * G::kBlocks][4];
    zero(ak);
    zero(av);
    for (int t = t0; t < t1; ++t) {
        ptx::cp_async_wait_group<0>();
        __syncthreads();
        fetch(t + 1);
        const int x = (t - t0) & 1;
        const uint32_t st = ring + (uint32_t)x * 2u * kTile;
        const float* sl = stat + x * 128;
        float s[4][4], dp[4][4];
        scores<D, 4>(sk, pair * 16, st, half * 32, lane, s);
        scores<D, 4>(sv, pair * 16, st + kTile, half * 32, lane, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int col = half * 32 + i * 8 + t4 * 2 + y;
                const float off = exponent_offset(sl[col]), dd = sl[64 + col];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p = on[h] ? ptx::ex2(fmaf(s[i][2 * h + y], c2, -off)) : 0.f;
                    s[i][2 * h + y] = p;
                    dp[i][2 * h + y] = p * (dp[i][2 * h + y] - dd);
                }
            }
        if constexpr (G::kExchange) {
            give(share, pair, half, lane, s);
            give(share + G::kShare, pair, half, lane, dp);
            __syncthreads();
            float f[8][4];
            take(share, pair, lane, f);
            accumulate<D, 8, G::kBlocks>(f, st + kTile, 0, half * G::kBlocks, lane, av);
            take(share + G::kShare, pair, lane, f);
            accumulate<D, 8, G::kBlocks>(f, st, 0, half * G::kBlocks, lane, ak);
        } else {
            accumulate<D, 4, 1>(s, st + kTile, half * 32, 0, lane, av);
            accumulate<D, 4, 1>(dp, st, half * 32, 0, lane, ak);
        }
    }
    ptx::cp_async_wait_all();
    allow_dependents();
    if constexpr (!G::kExchange) {
        join_pair(share, pair, half, lane, ak);
        join_pair(share + G::kShare, pair, half, lane, av);
        if (half == 1) return;
    }
    const size_t elems = (size_t)g.B * g.Lk * g.kv_heads * D;
    float* ok = splits > 1 ? parts + (size_t)split * 2 * elems : dk;
    float* ov = splits > 1 ? ok + elems : dv;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int key = kt * 64 + pair * 16 + h * 8 + gq;
        if (key >= g.Lk) continue;
        if (!on[h]) {  // an infinite gradient times its P of zero has made these sums NaN
#pragma unroll
            for (int i = 0; i < 4 * G::kBlocks; ++i) ak[i][2 * h] = ak[i][2 * h + 1] = av[i][2 * h] = av[i][2 * h + 1] = 0.f;
        }
        const size_t at = (((size_t)b * g.Lk + key) * g.kv_heads + j) * D + half * G::kBlocks * 32;
        store_row(ok + at, ak, h, g.scale, t4);
        store_row(ov + at, av, h, 1.f, t4);
    }
}

template <int D, int WM, int WN>
bra_status launch_forward(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o,
                          float* lse, CrossParts parts, cudaStream_t stream) {
    using S = Fwd<D, WM, WN>;
    auto* kernel = bra_cross_tf32_kernel<D, WM, WN>;
    if (!allow_shared<bra_cross_tf32_kernel<D, WM, WN>>(S::kBytes)) return BRA_ERR_CUDA;
    const int row_tiles = (g.rows + S::kRows - 1) / S::kRows;
    const long long grid = (long long)row_tiles * splits * g.kv_heads * g.B;
    if (grid > 0x7fffffffLL) return BRA_ERR_UNSUPPORTED;
    const cudaError_t e =
        launch_after_previous(kernel, dim3((unsigned)grid), dim3(S::kThreads), S::kBytes, stream,
                              static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v),
                              static_cast<float*>(o), lse, parts, g, row_tiles, splits);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

template <int D>
bra_status forward_d(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o, float* lse,
                     CrossParts parts, cudaStream_t stream) {
    return g.rows <= 16 ? launch_forward<D, 1, 4>(g, splits, q, k, v, o, lse, parts, stream)
                        : launch_forward<D, 4, 1>(g, splits, q, k, v, o, lse, parts, stream);
}

template <int D>
bra_status backward_d(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, const void* o,
                      const float* lse, const void* go, void* dq, void* dk, void* dv, float* delta, float* parts,
                      cudaStream_t stream) {
    using T = float;
    if (!allow_shared<bra_cross_tf32_dq_kernel<D>>(Grad<D>::kBytes) || !allow_shared<bra_cross_tf32_dkv_kernel<D>>(Grad<D>::kBytes))
        return BRA_ERR_CUDA;
    const int row_tiles = (g.rows + 63) / 64, key_tiles = (g.Lk + 63) / 64;
    const long long grid_q = (long long)row_tiles * g.kv_heads * g.B;
    const long long grid_k = (long long)key_tiles * splits * g.kv_heads * g.B;
    if (grid_q > 0x7fffffffLL || grid_k > 0x7fffffffLL) return BRA_ERR_UNSUPPORTED;
    cudaError_t e = launch_after_previous(bra_cross_tf32_dq_kernel<D>, dim3((unsigned)grid_q), dim3(kThreads),
                                          Grad<D>::kBytes, stream, (const T*)q, (const T*)k, (const T*)v, (const T*)o,
                                          lse, (const T*)go, (T*)dq, delta, g, row_tiles);
    if (e != cudaSuccess) return BRA_ERR_CUDA;
    if (grid_k == 0) return BRA_OK;
    e = launch_after_previous(bra_cross_tf32_dkv_kernel<D>, dim3((unsigned)grid_k), dim3(kThreads), Grad<D>::kBytes,
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
