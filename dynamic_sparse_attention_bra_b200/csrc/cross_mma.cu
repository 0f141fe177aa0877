// Cross attention to an encoder's states, bf16, on warp-level tensor-core
// products.  For every row r of a state head's group (a query token and one
// of the group's heads), over the valid states j of its batch entry:
//   s_j = scale <q_r, k_j>,  O_r = sum_j 2^(s'_j - m) v_j / sum_j 2^(s'_j - m),
// s' = s log2(e), m the running maximum of s': one pass over the states, the
// sums rescaled by 2^(old m - new m) when m grows.
//
// A CTA owns 16 MI WM rows of one (entry, state head) and streams the states
// in tiles of 64 through a ring of shared-memory stages (16-byte cp.async;
// rows that are padding or masked are filled with zeros, so that whatever is
// stored there never reaches a product).  WM warps share the rows and WN
// warps the states of a tile: many rows take WN = 1; few rows (single tokens)
// take WM = 1, WN = 4, whose four partial results are joined at the end.
// Where rows alone do not fill the GPU the states are split over CTAs too
// (``splits``) and a second kernel joins the parts, in a fixed order.
// Scores, maxima and sums are fp32; P is rounded once to bf16, an operand of
// the second product, while its sum keeps the unrounded values.
#include "cross_tile.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;
using wmma16::mma16816;

template <int D>
struct Ring {
    static constexpr uint32_t kTile = 64u * D * 2u;
    static constexpr int kStages = 3;
};

template <int D, int WM, int WN, int MI>
struct Smem {
    static constexpr int kRows = 16 * MI * WM;
    static constexpr uint32_t kQ = (uint32_t)kRows * D * 2u;
    static constexpr uint32_t kRing = Ring<D>::kStages * 2u * Ring<D>::kTile;
    // the join of WN warps reuses the ring: WN x rows x (d + 2) floats
    static constexpr uint32_t kJoin = WN > 1 ? (uint32_t)WN * kRows * (D + 2) * 4u : 0u;
    static constexpr uint32_t kBits = 2u * ValidBits::kWords * 4u;
    static constexpr uint32_t kBytes = kQ + (kRing > kJoin ? kRing : kJoin) + kBits;
};

template <int D, int WM, int WN, int MI>
__global__ void __launch_bounds__(32 * WM * WN)
bra_cross_mma_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                     const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                     CrossParts parts, CrossGeom g, int row_tiles, int splits) {
    using S = Smem<D, WM, WN, MI>;
    constexpr int kThreads = 32 * WM * WN, kStages = Ring<D>::kStages;
    constexpr int KW = 64 / WN;  // states of a tile that one warp takes
    constexpr int NT = KW / 8, KK = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sq = ptx::smem_addr(smem), ring = sq + S::kQ;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wm = warp % WM, wn = warp / WM;

    int id = blockIdx.x;
    const int tile = id % row_tiles;
    id /= row_tiles;
    const int split = id % splits;
    id /= splits;
    const int j = id % g.kv_heads, b = id / g.kv_heads;
    const int row0 = tile * S::kRows;

    grid_dependency_wait();
    const int n = cross_len(g, b);
    const int all_tiles = (n + 63) / 64, per = (all_tiles + splits - 1) / splits;
    const int t0 = split * per, t1 = min(all_tiles, t0 + per);
    ValidBits bits{reinterpret_cast<uint32_t*>(smem + S::kBytes - S::kBits),
                   g.kv_mask ? g.kv_mask + (size_t)b * g.Lk : nullptr, n};
    const __nv_bfloat16* kb = k + (size_t)b * g.k_batch + (size_t)j * D;
    const __nv_bfloat16* vb = v + (size_t)b * g.v_batch + (size_t)j * D;

    // Q rows (past the last: zeros, their results are not written)
    for (int e = threadIdx.x; e < S::kRows * (D / 8); e += kThreads) {
        const int r = e / (D / 8), c = e % (D / 8);
        const bool on = row0 + r < g.rows;
        ptx::cp_async16_zfill(sq + tile_offset<D>(r, c), on ? q + cross_q_offset(g, b, j, row0 + r) + c * 8 : q,
                              on ? 16u : 0u);
    }
    auto fetch = [&](int t) {
        if (t < t1) {
            bits.reach(t, t0, kThreads);
            const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
            const uint32_t st = ring + (uint32_t)((t - t0) % kStages) * 2u * Ring<D>::kTile;
            load_states<D, kThreads>(st, kb, g.k_row, t, w0, w1);
            load_states<D, kThreads>(st + Ring<D>::kTile, vb, g.v_row, t, w0, w1);
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(t0 + i);
    ptx::cp_async_wait_group<kStages - 2>();
    __syncthreads();

    uint32_t qa[MI][KK][4];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) frag_a<D>(sq, (wm * MI + mi) * 16, kk, lane, qa[mi][kk]);

    const float sl = g.scale * kLog2e;
    float acc[MI][D / 8][4], m[MI][2], l[MI][2];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mi][i][e] = 0.f;
        m[mi][0] = m[mi][1] = -INFINITY;
        l[mi][0] = l[mi][1] = 0.f;
    }

    for (int t = t0; t < t1; ++t) {
        if (t > t0) {
            ptx::cp_async_wait_group<kStages - 2>();
            __syncthreads();
        }
        fetch(t + kStages - 1);
        const uint32_t st = ring + (uint32_t)((t - t0) % kStages) * 2u * Ring<D>::kTile;
        const uint32_t w0 = bits.word(t, 0), w1 = bits.word(t, 1);
        if ((w0 | w1) == 0u) continue;
        float s[MI][NT][4];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mi][i][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int i = 0; i < NT; i += 2) {
                uint32_t bf[4];
                frag_nt<D>(st, wn * KW + i * 8, kk, lane, bf);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    mma16816(s[mi][i], qa[mi][kk][0], qa[mi][kk][1], qa[mi][kk][2], qa[mi][kk][3], bf[0], bf[1]);
                    mma16816(s[mi][i + 1], qa[mi][kk][0], qa[mi][kk][1], qa[mi][kk][2], qa[mi][kk][3], bf[2], bf[3]);
                }
            }
        if ((w0 & w1) != 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int c = wn * KW + i * 8 + (lane & 3) * 2;  // this thread's columns c, c + 1
                const uint32_t w = (c < 32 ? w0 : w1) >> (c & 31);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    if (!(w & 1u)) s[mi][i][0] = s[mi][i][2] = -INFINITY;
                    if (!(w & 2u)) s[mi][i][1] = s[mi][i][3] = -INFINITY;
                }
            }
        }
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < NT; ++i) mx = fmaxf(mx, fmaxf(s[mi][i][2 * h], s[mi][i][2 * h + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[mi][h], mx * sl);
                const float mu = mn == -INFINITY ? 0.f : mn;  // a row that has met no valid state yet
                const float alpha = ptx::ex2(m[mi][h] - mu);
                m[mi][h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 2 * h; e < 2 * h + 2; ++e) {
                        s[mi][i][e] = ptx::ex2(fmaf(s[mi][i][e], sl, -mu));
                        sum += s[mi][i][e];
                    }
                l[mi][h] = fmaf(l[mi][h], alpha, sum);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    acc[mi][i][2 * h] *= alpha;
                    acc[mi][i][2 * h + 1] *= alpha;
                }
            }
#pragma unroll
        for (int kt = 0; kt < KW / 16; ++kt) {
            uint32_t pa[MI][4];
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    pa[mi][x] = ptx::pack_bf16x2(s[mi][2 * kt + (x >> 1)][2 * (x & 1)],
                                                 s[mi][2 * kt + (x >> 1)][2 * (x & 1) + 1]);
#pragma unroll
            for (int c = 0; c < D / 8; c += 2) {
                uint32_t bf[4];
                frag_nn<D>(st + Ring<D>::kTile, wn * KW + kt * 16, c, lane, bf);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    mma16816(acc[mi][c], pa[mi][0], pa[mi][1], pa[mi][2], pa[mi][3], bf[0], bf[1]);
                    mma16816(acc[mi][c + 1], pa[mi][0], pa[mi][1], pa[mi][2], pa[mi][3], bf[2], bf[3]);
                }
            }
        }
    }
    ptx::cp_async_wait_all();
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[mi][h] += __shfl_xor_sync(0xffffffffu, l[mi][h], 1);
            l[mi][h] += __shfl_xor_sync(0xffffffffu, l[mi][h], 2);
        }
    allow_dependents();

    if constexpr (WN > 1) {
        // Join of the WN warps' parts through the ring's memory.
        float* jo = reinterpret_cast<float*>(smem + S::kQ);  // [WN][rows][D]
        float* jm = jo + WN * S::kRows * D;                  // [WN][rows][2]
        __syncthreads();
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = (wm * MI + mi) * 16 + h * 8 + (lane >> 2);
                float* row = jo + (size_t)(wn * S::kRows + r) * D + (lane & 3) * 2;
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2*>(row + i * 8) = make_float2(acc[mi][i][2 * h], acc[mi][i][2 * h + 1]);
                if ((lane & 3) == 0) {
                    jm[(wn * S::kRows + r) * 2] = m[mi][h];
                    jm[(wn * S::kRows + r) * 2 + 1] = l[mi][h];
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
                uint2 w;
                w.x = ptx::pack_bf16x2(x.x * inv, x.y * inv);
                w.y = ptx::pack_bf16x2(x.z * inv, x.w * inv);
                *reinterpret_cast<uint2*>(o + cross_o_offset(g, b, j, row0 + r) + c) = w;
                if (c == 0 && lse)
                    lse[cross_lse_offset(g, b, j, row0 + r)] = log_sum(mm, ll);
            }
        }
    } else {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row0 + (wm * MI + mi) * 16 + h * 8 + (lane >> 2);
                if (r >= g.rows) continue;
                const float ll = l[mi][h];
                if (splits > 1) {
                    const size_t at = ((size_t)(split * g.B + b) * g.kv_heads + j) * g.rows + r;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        *reinterpret_cast<float2*>(parts.o + at * D + i * 8 + (lane & 3) * 2) =
                            make_float2(acc[mi][i][2 * h], acc[mi][i][2 * h + 1]);
                    if ((lane & 3) == 0) parts.ml[at] = make_float2(m[mi][h], ll);
                } else {
                    const float inv = inverse_sum(ll);
                    __nv_bfloat16* row = o + cross_o_offset(g, b, j, r) + (lane & 3) * 2;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        *reinterpret_cast<uint32_t*>(row + i * 8) =
                            ptx::pack_bf16x2(acc[mi][i][2 * h] * inv, acc[mi][i][2 * h + 1] * inv);
                    if ((lane & 3) == 0 && lse)
                        lse[cross_lse_offset(g, b, j, r)] = log_sum(m[mi][h], ll);
                }
            }
    }
}

// Joins the parts of a split, in the order of the splits: thread = 4 channels of a row.
template <typename T>
__global__ void __launch_bounds__(128)
bra_cross_join_kernel(CrossParts parts, T* __restrict__ o, float* __restrict__ lse, CrossGeom g, int splits,
                      long long rows_all) {
    const int per = g.d / 4;  // threads of a row
    const long long at = (long long)blockIdx.x * (128 / per) + threadIdx.x / per;
    const int c = (threadIdx.x % per) * 4;
    grid_dependency_wait();
    allow_dependents();
    if (at >= rows_all) return;
    float m = -INFINITY, l = 0.f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) m = fmaxf(m, __ldcg(parts.ml + s * rows_all + at).x);
    const float mu = m == -INFINITY ? 0.f : m;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        const float2 ml = __ldcg(parts.ml + s * rows_all + at);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(parts.o + (size_t)(s * rows_all + at) * g.d + c));
        const float f = ptx::ex2(ml.x - mu);
        l = fmaf(ml.y, f, l);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
    }
    const int r = (int)(at % g.rows);
    const long long bj = at / g.rows;
    const int j = (int)(bj % g.kv_heads), b = (int)(bj / g.kv_heads);
    const float inv = inverse_sum(l);
    T* row = o + cross_o_offset(g, b, j, r) + c;
    row[0] = from_f32<T>(x.x * inv);
    row[1] = from_f32<T>(x.y * inv);
    row[2] = from_f32<T>(x.z * inv);
    row[3] = from_f32<T>(x.w * inv);
    if (c == 0 && lse) lse[cross_lse_offset(g, b, j, r)] = log_sum(m, l);
}

template <int D, int WM, int WN, int MI>
bra_status launch(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o, float* lse,
                  CrossParts parts, cudaStream_t stream) {
    using S = Smem<D, WM, WN, MI>;
    auto* kernel = bra_cross_mma_kernel<D, WM, WN, MI>;
    if (!allow_shared<bra_cross_mma_kernel<D, WM, WN, MI>>(S::kBytes)) return BRA_ERR_CUDA;
    const int row_tiles = (g.rows + S::kRows - 1) / S::kRows;
    const long long grid = (long long)row_tiles * splits * g.kv_heads * g.B;
    if (grid > 0x7fffffffLL) return BRA_ERR_UNSUPPORTED;
    const cudaError_t e = launch_after_previous(
        kernel, dim3((unsigned)grid), dim3(32 * WM * WN), S::kBytes, stream, static_cast<const __nv_bfloat16*>(q),
        static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(o),
        lse, parts, g, row_tiles, splits);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

template <int D>
bra_status launch_d(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o, float* lse,
                    CrossParts parts, cudaStream_t stream) {
    if (g.rows <= 16) return launch<D, 1, 4, 1>(g, splits, q, k, v, o, lse, parts, stream);
    constexpr int kMI = D == 32 ? 2 : 1;
    return launch<D, 4, 1, kMI>(g, splits, q, k, v, o, lse, parts, stream);
}

int rows_per_cta(const CrossGeom& g, bool bf16) {
    if (!bf16) return g.rows <= 16 ? 16 : 64;
    if (cross_tc_covers(g)) return cross_tc_rows(g);
    return g.rows <= 16 ? 16 : (g.d == 32 ? 128 : 64);
}

}  // namespace

// The states are split where (row tiles x state heads x entries) leave SMs
// idle: enough parts for eight small CTAs on each SM (of which four run: entries
// of different lengths even out; four parts: 81 us where eight take 76, sixteen
// 82: 16 entries of up to 16384 states, 8 heads of 64), none below 256 states.  The
// many-row form takes one CTA on an SM and parts of 128 states and more (2 x 4096 rows
// of 64 over 1024 states: 17 us for 20 with parts of 512); at most 16, for the join
// reads them all (128 rows of 32 over 8192: 20 us with 16 parts, 35 with 64); none
// below 1024, where the parts' traffic costs more (64 x 256 rows of 128 over 512: 17 us
// whole, 23 in two).
CrossPlan cross_forward_plan(const CrossGeom& g, bool bf16) {
    CrossPlan p{1};
    const int sms = sm_count();
    if (sms <= 0 || g.Lk < 512) return p;
    const int rpc = rows_per_cta(g, bf16);
    const long long ctas = (long long)((g.rows + rpc - 1) / rpc) * g.kv_heads * g.B;
    const bool tc = bf16 && cross_tc_covers(g);
    if (ctas <= 0 || ctas >= (tc ? 1LL : 2LL) * sms) return p;
    long long s = (tc ? 1LL : 8LL) * sms / ctas;
    const long long most = tc ? (g.Lk < 1024 ? 1 : g.Lk < 2048 ? g.Lk / 128 : 16) : g.Lk / 256;
    if (s > most) s = most;
    p.splits = s < 1 ? 1 : (int)s;
    return p;
}

size_t cross_forward_part_rows(const CrossGeom& g, const CrossPlan& p) {
    return p.splits > 1 ? (size_t)p.splits * g.B * g.kv_heads * g.rows : 0;
}

bra_status cross_forward_bf16(const CrossGeom& g, const CrossPlan& p, const void* q, const void* k, const void* v,
                              void* o, float* lse, CrossParts parts, int* status, cudaStream_t stream) {
    if (cross_short_covers(g)) return cross_forward_short(g, q, k, v, o, lse, stream);
    const bra_status rc = cross_tc_covers(g) ? cross_forward_tc(g, p.splits, q, k, v, o, lse, parts, status, stream)
                          : g.d == 32   ? launch_d<32>(g, p.splits, q, k, v, o, lse, parts, stream)
                          : g.d == 64 ? launch_d<64>(g, p.splits, q, k, v, o, lse, parts, stream)
                                      : launch_d<128>(g, p.splits, q, k, v, o, lse, parts, stream);
    if (rc != BRA_OK || p.splits == 1) return rc;
    return cross_join(g, p.splits, true, parts, o, lse, stream);
}

bra_status cross_join(const CrossGeom& g, int splits, bool bf16, CrossParts parts, void* o, float* lse,
                      cudaStream_t stream) {
    const long long rows = (long long)g.B * g.kv_heads * g.rows;
    const int per_cta = 128 / (g.d / 4);
    const long long grid = (rows + per_cta - 1) / per_cta;
    if (grid > 0x7fffffffLL) return BRA_ERR_UNSUPPORTED;
    const cudaError_t e =
        bf16 ? launch_after_previous(bra_cross_join_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(128), 0, stream,
                                     parts, static_cast<__nv_bfloat16*>(o), lse, g, splits, rows)
             : launch_after_previous(bra_cross_join_kernel<float>, dim3((unsigned)grid), dim3(128), 0, stream, parts,
                                     static_cast<float*>(o), lse, g, splits, rows);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace bra
