// Gradients of the cross attention, bf16, on tcgen05 tensor cores: the form
// for many rows.  The mathematics, and the split into a kernel for dQ and D
// and one for dK and dV, are those of cross_backward.cu.
//
// Both kernels have one shape: a tile of 128 rows (of Q and dO; of K and V)
// stays in shared memory while blocks of 64 columns (of K and V; of Q and dO)
// stream past.  Per block S = R1 C1^T and dP = R2 C2^T land in TMEM; a thread
// per row forms P = 2^(s - lse) and dS = P (dP - D), rounds each once to bf16
// and writes them over the scores that it has read; then they are the TMEM
// operands of
//   dQ += dS K,   sum_j P_j k_j += P K      (rows of queries)
//   dK += dS Q,   dV += P dO                (rows of states)
// whose sums stay in TMEM over all blocks.
//
// A unit is two tiles (one at d = 128: its sums take 256 of the 512 columns)
// that share the streamed blocks; while one tile's products run, the other's
// threads have the exponentials.  Roles of the warps: 0, 1 issue the products
// of tile 0, 1; 2 loads (TMA; tiles and blocks with a masked or missing state by
// cp.async, those rows filled with zeros); 3-6, 7-10 have a row a thread.
// Every mbarrier wait is bounded; on expiry the kernel records kDevTimeout, stops
// all roles, drains its products and frees TMEM.
#include "cross_tc.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;

constexpr int kCtrl = 3;
constexpr int kStages = 4;  // at most
constexpr int BN = 64;      // columns of a block

struct Barriers {
    uint64_t c_full[kStages], c_empty[kStages];
    uint64_t r_full[2][2], r_empty[2][2];  // [tile][buffer]
    uint64_t s_full[2], p_full[2], acc_done[2], drain[2];
    uint32_t words[kStages][2];  // dQ: the block's valid states, where a mask says which
    uint32_t tmem;
    int abort;
};

template <int D>
struct Cfg {
    static constexpr int kTiles = D == 128 ? 1 : 2;
    static constexpr int kThreads = 32 * (kCtrl + 4 * kTiles);
    static constexpr uint32_t kTileCols = 256;  // TMEM columns from tile to tile
    static constexpr uint32_t kDp = 64, kAcc1 = 128, kAcc2 = 128 + D;
    static constexpr uint32_t kRow = 128u * D * 2u, kCol = (uint32_t)BN * D * 2u;
    static constexpr int kRing = D == 128 ? 3 : 4;
    // rows [tile][buffer] x (R1 | R2), then stages of C1 | C2, the columns' statistics, barriers
    static constexpr uint32_t kOffCol = kTiles * 2 * 2 * kRow;
    static constexpr uint32_t kOffStat = kOffCol + kRing * 2 * kCol;
    static constexpr uint32_t kOffBar = kOffStat + kRing * 2 * BN * 4;
    static constexpr uint32_t kSmem = kOffBar + (uint32_t)sizeof(Barriers) + 1024u;
};

struct BwdPlan {
    int groups;         // units of kTiles x 128 rows in a (entry, state head)
    int splits;         // dK, dV: parts of the rows of queries
    int units;
    int tma_r, tma_c;   // loads by TMA (the maps could be made)
};

struct Unit {
    int b, j, row0, split, n, t0, nb;  // first block and number of blocks
};

template <bool STATES, int TILE_ROWS>
__device__ __forceinline__ Unit unit_at(const CrossGeom& g, const BwdPlan& p, int u) {
    Unit x;
    x.row0 = (u % p.groups) * TILE_ROWS;
    u /= p.groups;
    x.split = u % p.splits;
    u /= p.splits;
    x.j = u % g.kv_heads;
    x.b = u / g.kv_heads;
    x.n = cross_len(g, x.b);
    if (STATES) {
        const int all = (g.rows + BN - 1) / BN, per = (all + p.splits - 1) / p.splits;
        x.t0 = x.split * per;
        x.nb = x.row0 < x.n ? max(0, min(all, x.t0 + per) - x.t0) : 0;
    } else {
        x.t0 = 0;
        x.nb = (x.n + BN - 1) / BN;
    }
    return x;
}

// Columns of block t that products see (dQ: its states, in steps of 16).
template <bool STATES>
__device__ __forceinline__ int block_cols(const Unit& x, int b) {
    return STATES ? BN : (min(BN, x.n - (x.t0 + b) * BN) + 15) & ~15;
}

// ``rows`` rows of queries (dense: O's layout) from row0; past the last: zeros.
template <int D>
__device__ __forceinline__ void load_queries(uint32_t dst, const __nv_bfloat16* base, bool dense, const CrossGeom& g,
                                             int b, int j, int row0, int rows, int lane) {
#pragma unroll 4
    for (int e = lane; e < rows * (D / 8); e += 32) {
        const int r = e / (D / 8), c = e % (D / 8);
        const bool on = row0 + r < g.rows;
        const size_t off = !on ? 0 : dense ? cross_o_offset(g, b, j, row0 + r) : cross_q_offset(g, b, j, row0 + r);
        ptx::cp_async16_zfill(dst + op_offset<D>(r, c, rows), base + off + (on ? c * 8 : 0), on ? 16u : 0u);
    }
}

// ``rows`` rows of states from key0; rows whose bit in w is off: zeros.
template <int D, int W>
__device__ __forceinline__ void load_states(uint32_t dst, const __nv_bfloat16* base, long long step, int key0,
                                            const uint32_t (&w)[W], int rows, int tile_rows, int lane) {
#pragma unroll 4
    for (int e = lane; e < rows * (D / 8); e += 32) {
        const int r = e / (D / 8), c = e % (D / 8);
        uint32_t word = w[0];
#pragma unroll
        for (int h = 1; h < W; ++h) word = r >= h * 32 ? w[h] : word;
        const bool on = (word >> (r & 31)) & 1u;
        ptx::cp_async16_zfill(dst + op_offset<D>(r, c, tile_rows), on ? base + (size_t)(key0 + r) * step + c * 8 : base,
                              on ? 16u : 0u);
    }
}

// Validity of 32 W states from key0 as bits; true if all are.
template <int W>
__device__ __forceinline__ bool valid_words(const CrossGeom& g, int b, int n, int key0, int lane, uint32_t (&w)[W]) {
    uint32_t every = 0xffffffffu;
#pragma unroll
    for (int h = 0; h < W; ++h) {
        const int key = key0 + h * 32 + lane;
        w[h] = __ballot_sync(0xffffffffu, key < n && (!g.kv_mask || __ldcg(g.kv_mask + (size_t)b * g.Lk + key) != 0));
        every &= w[h];
    }
    return every == 0xffffffffu;
}

// STATES: the rows are states (dK, dV), the columns queries; else the rows are
// queries (dQ), the columns states.
template <int D, bool STATES>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
bra_cross_tc_backward_kernel(const __grid_constant__ CUtensorMap tr1, const __grid_constant__ CUtensorMap tr2,
                             const __grid_constant__ CUtensorMap tc1, const __grid_constant__ CUtensorMap tc2,
                             const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                             const __nv_bfloat16* o, const float* lse, const __nv_bfloat16* go, __nv_bfloat16* out1,
                             __nv_bfloat16* out2, float* delta, float* parts, CrossGeom g, BwdPlan p, int* status) {
    using C = Cfg<D>;
    constexpr int kRing = C::kRing, kTileRows = 128 * C::kTiles;
    constexpr int kPanels = D == 128 ? 2 : 1;  // of 64 channels (D = 32: one of 32)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    Barriers* sb = reinterpret_cast<Barriers*>(smem + C::kOffBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(&sb->c_full[i], 1);
            ptx::mbar_init(&sb->c_empty[i], C::kTiles);
        }
        for (int x = 0; x < 2; ++x) {
            for (int y = 0; y < 2; ++y) {
                ptx::mbar_init(&sb->r_full[x][y], 1);
                ptx::mbar_init(&sb->r_empty[x][y], STATES ? 1 : 1 + 128);  // the products; the reads of dO for D
            }
            ptx::mbar_init(&sb->s_full[x], 1);
            ptx::mbar_init(&sb->p_full[x], 128);
            ptx::mbar_init(&sb->acc_done[x], 1);
            ptx::mbar_init(&sb->drain[x], 1);
        }
        sb->abort = 0;
        ptx::mbar_init_fence();
    }
    if (warp == 0) {
        ptx::tmem_alloc(&sb->tmem, 512);
        ptx::tmem_relinquish();
        ptx::tc_fence_before();
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sb->tmem;
    grid_dependency_wait();

    if (warp < 2) {
        // ------------------------------------------------ products of tile ``warp``
        if (lane == 0 && warp < C::kTiles) {
            const int grp = warp;
            const uint32_t cols = tmem + (uint32_t)grp * C::kTileCols;
            const uint32_t idesc_acc = ptx::idesc_bf16_f32(128, D, false, true);
            int i = 0, use = 0;  // blocks and units so far
            bool ok = true;
            for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const Unit x = unit_at<STATES, kTileRows>(g, p, u);
                if (x.nb == 0) continue;
                ok = wait_or_abort(&sb->r_full[grp][use & 1], (use >> 1) & 1, &sb->abort, status);
                const uint32_t r1 = sbase + (uint32_t)(grp * 2 + (use & 1)) * 2u * C::kRow;
                for (int b = 0; ok && b < x.nb; ++b, ++i) {
                    const int stage = i % kRing;
                    const uint32_t c1 = sbase + C::kOffCol + (uint32_t)stage * 2u * C::kCol;
                    // the columns of S and dP hold the last block's P and dS until their products end
                    if (!wait_or_abort(&sb->c_full[stage], (i / kRing) & 1, &sb->abort, status) ||
                        (i > 0 && !wait_or_abort(&sb->acc_done[grp], (i - 1) & 1, &sb->abort, status))) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const int nc = block_cols<STATES>(x, b);
                    const uint32_t idesc = ptx::idesc_bf16_f32(128, nc, false, false);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        ptx::mma_bf16(cols, k_major<D>(r1, kk, 128), k_major<D>(c1, kk, BN), idesc, kk);
                        ptx::mma_bf16(cols + C::kDp, k_major<D>(r1 + C::kRow, kk, 128), k_major<D>(c1 + C::kCol, kk, BN),
                                      idesc, kk);
                    }
                    ptx::mma_commit(&sb->s_full[grp]);
                    if (b == x.nb - 1) ptx::mma_commit(&sb->r_empty[grp][use & 1]);
                    if (!wait_or_abort(&sb->p_full[grp], i & 1, &sb->abort, status)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t c_acc2 = STATES ? c1 + C::kCol : c1;
                    for (int kk = 0; kk < (nc >> 4); ++kk) {
                        ptx::mma_bf16_ta(cols + C::kAcc1, cols + C::kDp + (uint32_t)kk * 8u, v_operand<D>(c1, kk, BN),
                                         idesc_acc, b > 0 || kk > 0);
                        ptx::mma_bf16_ta(cols + C::kAcc2, cols + (uint32_t)kk * 8u, v_operand<D>(c_acc2, kk, BN),
                                         idesc_acc, b > 0 || kk > 0);
                    }
                    ptx::mma_commit(&sb->acc_done[grp]);
                    ptx::mma_commit(&sb->c_empty[stage]);
                }
                ++use;
            }
            ptx::mma_commit(&sb->drain[grp]);
            ptx::mbar_wait(&sb->drain[grp], 0, kWait);
        }
        __syncwarp();
    } else if (warp < kCtrl) {
        // ------------------------------------------------------------------ loads
        if (lane == 0) {
            ptx::tma_prefetch_desc(&tr1);
            ptx::tma_prefetch_desc(&tr2);
            ptx::tma_prefetch_desc(&tc1);
            ptx::tma_prefetch_desc(&tc2);
        }
        int i = 0, use = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<STATES, kTileRows>(g, p, u);
            if (x.nb == 0) continue;
            const __nv_bfloat16* kbase = k + (size_t)x.b * g.k_batch + (size_t)x.j * D;
            const __nv_bfloat16* vbase = v + (size_t)x.b * g.v_batch + (size_t)x.j * D;
            // TMA of one box of states (rows from key0) or queries (rows from r0), R or C operands
            auto tma_states = [&](uint32_t dst, uint32_t second, const CUtensorMap* m1, const CUtensorMap* m2, int key0,
                                  uint32_t rows, uint64_t* full) {
                ptx::mbar_arrive_expect_tx(full, 2u * rows * D * 2u);
#pragma unroll
                for (int c = 0; c < kPanels; ++c) {
                    ptx::tma_load_4d(dst + (uint32_t)c * rows * 128u, m1, c * 64, x.j, key0, g.k_batch ? x.b : 0, full);
                    ptx::tma_load_4d(dst + second + (uint32_t)c * rows * 128u, m2, c * 64, x.j, key0,
                                     g.v_batch ? x.b : 0, full);
                }
            };
            auto tma_queries = [&](uint32_t dst, uint32_t second, const CUtensorMap* m1, const CUtensorMap* m2, int r0,
                                   uint32_t rows, uint64_t* full) {
                ptx::mbar_arrive_expect_tx(full, 2u * rows * D * 2u);
#pragma unroll
                for (int c = 0; c < kPanels; ++c) {
                    ptx::tma_load_4d(dst + (uint32_t)c * rows * 128u, m1, c * 64, x.j * g.rep, r0 / g.rep,
                                     g.q_batch ? x.b : 0, full);
                    ptx::tma_load_4d(dst + second + (uint32_t)c * rows * 128u, m2, c * 64, x.j * g.rep, r0 / g.rep, x.b,
                                     full);
                }
            };
            auto landed = [&](uint64_t* full) {  // this warp's cp.async and stores, seen by the products
                ptx::cp_async_wait_all();
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(full);
            };
            for (int grp = 0; grp < C::kTiles; ++grp) {
                uint64_t* full = &sb->r_full[grp][use & 1];
                if (use >= 2 && !warp_wait(&sb->r_empty[grp][use & 1], ((use >> 1) - 1) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                const uint32_t r1 = sbase + (uint32_t)(grp * 2 + (use & 1)) * 2u * C::kRow;
                const int row0 = x.row0 + grp * 128;
                if constexpr (STATES) {
                    uint32_t w[4];
                    if (valid_words(g, x.b, x.n, row0, lane, w) && p.tma_r) {
                        if (lane == 0) tma_states(r1, C::kRow, &tr1, &tr2, row0, 128, full);
                    } else {
                        load_states<D>(r1, kbase, g.k_row, row0, w, 128, 128, lane);
                        load_states<D>(r1 + C::kRow, vbase, g.v_row, row0, w, 128, 128, lane);
                        landed(full);
                    }
                } else {
                    if (p.tma_r) {
                        if (lane == 0) tma_queries(r1, C::kRow, &tr1, &tr2, row0, 128, full);
                    } else {
                        load_queries<D>(r1, q, false, g, x.b, x.j, row0, 128, lane);
                        load_queries<D>(r1 + C::kRow, go, true, g, x.b, x.j, row0, 128, lane);
                        landed(full);
                    }
                }
            }
            float st[4];  // STATES: this lane's share of the next block's log sums (2) and D (2)
            auto read_stats = [&](int b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (x.t0 + b) * BN + h * 32 + lane;
                    const bool in = b < x.nb && r < g.rows;
                    const size_t at = in ? cross_lse_offset(g, x.b, x.j, r) : 0;
                    st[h] = in ? __ldcg(lse + at) : -INFINITY;
                    st[2 + h] = in ? __ldcg(delta + at) : 0.f;
                }
            };
            if (STATES) read_stats(0);
            for (int b = 0; ok && b < x.nb; ++b, ++i) {
                const int stage = i % kRing, t = x.t0 + b;
                uint32_t w[2];
                const bool whole = STATES || valid_words(g, x.b, x.n, t * BN, lane, w);
                if (i >= kRing && !warp_wait(&sb->c_empty[stage], ((i / kRing) - 1) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                const uint32_t c1 = sbase + C::kOffCol + (uint32_t)stage * 2u * C::kCol;
                uint64_t* full = &sb->c_full[stage];
                if constexpr (STATES) {
                    float* stat = reinterpret_cast<float*>(smem + C::kOffStat) + stage * 2 * BN;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        stat[h * 32 + lane] = -exponent_offset(st[h]);
                        stat[BN + h * 32 + lane] = -st[2 + h];
                    }
                    __syncwarp();
                    if (p.tma_c) {
                        if (lane == 0) tma_queries(c1, C::kCol, &tc1, &tc2, t * BN, BN, full);
                    } else {
                        load_queries<D>(c1, q, false, g, x.b, x.j, t * BN, BN, lane);
                        load_queries<D>(c1 + C::kCol, go, true, g, x.b, x.j, t * BN, BN, lane);
                        landed(full);
                    }
                    read_stats(b + 1);
                } else {
                    if (lane == 0 && g.kv_mask) {
                        sb->words[stage][0] = w[0];
                        sb->words[stage][1] = w[1];
                    }
                    if (whole && p.tma_c) {
                        if (lane == 0) tma_states(c1, C::kCol, &tc1, &tc2, t * BN, BN, full);
                    } else {
                        const int rows = block_cols<false>(x, b);  // no product reads past them
                        load_states<D>(c1, kbase, g.k_row, t * BN, w, rows, BN, lane);
                        load_states<D>(c1 + C::kCol, vbase, g.v_row, t * BN, w, rows, BN, lane);
                        landed(full);
                    }
                }
            }
            ++use;
        }
    } else {
        // ---------------------------------------------------- P, dS and the epilogue
        const int grp = (warp - kCtrl) >> 2, qd = warp & 3;
        const int row = 32 * qd + lane;
        const uint32_t cols = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)grp * C::kTileCols;
        const float c2 = g.scale * kLog2e;
        int i = 0, use = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<STATES, kTileRows>(g, p, u);
            const int r0 = x.row0 + grp * 128 + row;
            const bool in = r0 < (STATES ? g.Lk : g.rows);
            float noff = -INFINITY, nd = 0.f, rest = 0.f;  // dQ: the row's -offset and -D0; sum of dS
            if (!STATES) {
                // D0 = <dO, O>: O from memory, dO from the tile
                float d0 = 0.f;
                const size_t off = in ? cross_o_offset(g, x.b, x.j, r0) : 0;
                uint4 ov[D / 8];
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    ov[c] = in ? __ldcg(reinterpret_cast<const uint4*>(o + off) + c) : make_uint4(0u, 0u, 0u, 0u);
                if (in) noff = -exponent_offset(__ldcg(lse + cross_lse_offset(g, x.b, x.j, r0)));
                if (x.nb > 0) {
                    if (!warp_wait(&sb->r_full[grp][use & 1], (use >> 1) & 1, &sb->abort, status)) break;
                    const uint8_t* r2 = smem + (size_t)(grp * 2 + (use & 1)) * 2 * C::kRow + C::kRow;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        float a[8], h[8];
                        unpack16(ov[c], a, (const __nv_bfloat16*)nullptr);
                        unpack16(*reinterpret_cast<const uint4*>(r2 + op_offset<D>(row, c, 128)), h,
                                 (const __nv_bfloat16*)nullptr);
#pragma unroll
                        for (int e = 0; e < 8; ++e) d0 = fmaf(a[e], h[e], d0);
                    }
                    ptx::mbar_arrive(&sb->r_empty[grp][use & 1]);
                }
                nd = -d0;
            }
            const uint64_t c22 = ptx::pack_f32x2(c2, c2);
            uint64_t rest2 = 0ull;
            for (int b = 0; b < x.nb; ++b, ++i) {
                const int stage = i % kRing;
                if (!warp_wait(&sb->s_full[grp], i & 1, &sb->abort, status) ||
                    ((STATES || g.kv_mask) && !warp_wait(&sb->c_full[stage], (i / kRing) & 1, &sb->abort, status))) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const int nc = block_cols<STATES>(x, b), left = x.n - (x.t0 + b) * BN;
                const float* stat = reinterpret_cast<const float*>(smem + C::kOffStat) + stage * 2 * BN;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!STATES && nc <= h * 32) break;
                    uint32_t s[32], dp[32];
                    ptx::tmem_load_pair(cols + h * 32, cols + C::kDp + h * 32, s, dp);
                    uint32_t w = 0xffffffffu;
                    if (!STATES) {
                        const int some = left - h * 32;
                        w = g.kv_mask ? sb->words[stage][h] : (some >= 32 ? 0xffffffffu : (1u << max(some, 0)) - 1u);
                    }
                    uint32_t pp[16], pd[16];
                    const uint64_t noff2 = ptx::pack_f32x2(noff, noff), nd2 = ptx::pack_f32x2(nd, nd);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        uint64_t no = noff2, dd = nd2;
                        if constexpr (STATES) {
                            no = *reinterpret_cast<const uint64_t*>(stat + h * 32 + 2 * e);
                            dd = *reinterpret_cast<const uint64_t*>(stat + BN + h * 32 + 2 * e);
                        }
                        float lo, hi;
                        ptx::unpack_f32x2(
                            ptx::fma_f32x2(ptx::pack_f32x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c22,
                                           no),
                            lo, hi);
                        lo = ptx::ex2(lo);
                        hi = ptx::ex2(hi);
                        uint64_t ds = ptx::mul_f32x2(
                            ptx::pack_f32x2(lo, hi),
                            ptx::add_f32x2(ptx::pack_f32x2(__uint_as_float(dp[2 * e]), __uint_as_float(dp[2 * e + 1])),
                                           dd));
                        float dlo, dhi;
                        ptx::unpack_f32x2(ds, dlo, dhi);
                        if (!STATES && w != 0xffffffffu) {  // (uniform) masked states: nothing, whatever the sums hold
                            if (!((w >> (2 * e)) & 1u)) lo = dlo = 0.f;
                            if (!((w >> (2 * e + 1)) & 1u)) hi = dhi = 0.f;
                            ds = ptx::pack_f32x2(dlo, dhi);
                        }
                        if (!STATES) rest2 = ptx::add_f32x2(rest2, ds);
                        pp[e] = ptx::pack_bf16x2(lo, hi);
                        pd[e] = ptx::pack_bf16x2(dlo, dhi);
                    }
                    ptx::tmem_st16(cols + h * 16, pp);
                    ptx::tmem_st16(cols + C::kDp + h * 16, pd);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&sb->p_full[grp]);
            }
            if (!ok) break;
            if (x.nb > 0) {
                if (!warp_wait(&sb->acc_done[grp], (i - 1) & 1, &sb->abort, status)) break;
                ptx::tc_fence_after();
                ++use;
            }
            bool live = x.nb > 0;
            size_t at = 0;
            if (STATES) {
                live = live && in && r0 < x.n && (!g.kv_mask || __ldcg(g.kv_mask + (size_t)x.b * g.Lk + r0) != 0);
                if (in) at = (((size_t)x.b * g.Lk + r0) * g.kv_heads + x.j) * D;
            } else {
                float lo, hi;
                ptx::unpack_f32x2(rest2, lo, hi);
                rest = lo + hi;
                if (in) {
                    at = cross_o_offset(g, x.b, x.j, r0);
                    delta[cross_lse_offset(g, x.b, x.j, r0)] = rest - nd;
                }
            }
            const size_t elems = (size_t)g.B * g.Lk * g.kv_heads * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t a1[32], a2[32];
                if (x.nb > 0) ptx::tmem_load_pair(cols + C::kAcc1 + c, cols + C::kAcc2 + c, a1, a2);
                if (!in) continue;
                float f1[32], f2[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    f1[e] = live ? __uint_as_float(a1[e]) : 0.f;
                    f2[e] = live ? __uint_as_float(a2[e]) : 0.f;
                    if (!STATES) f1[e] = fmaf(-rest, f2[e], f1[e]);
                    f1[e] *= g.scale;
                }
                if (STATES && p.splits > 1) {
                    float* out = parts + (size_t)x.split * 2 * elems + at + c;
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        *reinterpret_cast<float4*>(out + e) = make_float4(f1[e], f1[e + 1], f1[e + 2], f1[e + 3]);
                        *reinterpret_cast<float4*>(out + elems + e) = make_float4(f2[e], f2[e + 1], f2[e + 2], f2[e + 3]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        *reinterpret_cast<uint4*>(out1 + at + c + e) =
                            make_uint4(ptx::pack_bf16x2(f1[e], f1[e + 1]), ptx::pack_bf16x2(f1[e + 2], f1[e + 3]),
                                       ptx::pack_bf16x2(f1[e + 4], f1[e + 5]), ptx::pack_bf16x2(f1[e + 6], f1[e + 7]));
                        if (STATES)
                            *reinterpret_cast<uint4*>(out2 + at + c + e) =
                                make_uint4(ptx::pack_bf16x2(f2[e], f2[e + 1]), ptx::pack_bf16x2(f2[e + 2], f2[e + 3]),
                                           ptx::pack_bf16x2(f2[e + 4], f2[e + 5]), ptx::pack_bf16x2(f2[e + 6], f2[e + 7]));
                    }
                }
            }
            ptx::tc_fence_before();  // the sums are read before the next tile's first products, which p_full orders after
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    allow_dependents();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Maps of Q and dO for boxes of ``rows`` rows; of K and V.
bool query_maps(CUtensorMap* a, CUtensorMap* b, const CrossGeom& g, const void* q, const void* go, int rows) {
    const long long width = (long long)g.heads * g.d;
    return rows % g.rep == 0 && g.Lq >= rows / g.rep &&
           encode_heads_map(a, q, g.B, g.Lq, g.heads, g.d, g.q_row, g.q_batch, rows / g.rep, g.rep) &&
           encode_heads_map(b, go, g.B, g.Lq, g.heads, g.d, width, width * g.Lq, rows / g.rep, g.rep);
}
bool state_maps(CUtensorMap* a, CUtensorMap* b, const CrossGeom& g, const void* k, const void* v, int rows) {
    return g.Lk >= rows && encode_heads_map(a, k, g.B, g.Lk, g.kv_heads, g.d, g.k_row, g.k_batch, rows, 1) &&
           encode_heads_map(b, v, g.B, g.Lk, g.kv_heads, g.d, g.v_row, g.v_batch, rows, 1);
}

template <int D, bool STATES>
bra_status launch(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, const void* o,
                  const float* lse, const void* go, void* out1, void* out2, float* delta, float* parts, int* status,
                  cudaStream_t stream) {
    using C = Cfg<D>;
    using T = __nv_bfloat16;
    BwdPlan p = {};
    const int tile_rows = 128 * C::kTiles, length = STATES ? g.Lk : g.rows;
    p.groups = (length + tile_rows - 1) / tile_rows;
    p.splits = STATES ? splits : 1;
    const long long units = (long long)p.groups * p.splits * g.kv_heads * g.B;
    if (units == 0) return BRA_OK;
    if (units > 0x3fffffffLL) return BRA_ERR_UNSUPPORTED;
    p.units = (int)units;
    CUtensorMap tr1 = {}, tr2 = {}, tc1 = {}, tc2 = {};
    if (STATES) {
        p.tma_r = state_maps(&tr1, &tr2, g, k, v, 128);
        p.tma_c = query_maps(&tc1, &tc2, g, q, go, BN);
    } else {
        p.tma_r = query_maps(&tr1, &tr2, g, q, go, 128);
        p.tma_c = state_maps(&tc1, &tc2, g, k, v, BN);
    }
    const int sms = sm_count();
    if (sms <= 0) return BRA_ERR_CUDA;
    auto* kernel = bra_cross_tc_backward_kernel<D, STATES>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
        return BRA_ERR_CUDA;
    const int grid = units < sms ? (int)units : sms;
    const cudaError_t e = launch_after_previous(kernel, dim3(grid), dim3(C::kThreads), C::kSmem, stream, tr1, tr2, tc1,
                                                tc2, (const T*)q, (const T*)k, (const T*)v, (const T*)o, lse,
                                                (const T*)go, (T*)out1, (T*)out2, delta, parts, g, p, status);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

template <int D>
bra_status launch_d(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, const void* o,
                    const float* lse, const void* go, void* dq, void* dk, void* dv, float* delta, float* parts,
                    int* status, cudaStream_t stream) {
    const bra_status rc =
        launch<D, false>(g, 1, q, k, v, o, lse, go, dq, nullptr, delta, nullptr, status, stream);
    if (rc != BRA_OK) return rc;
    return launch<D, true>(g, splits, q, k, v, o, lse, go, dk, dv, delta, parts, status, stream);
}

}  // namespace

bool cross_tc_backward_covers(const CrossGeom& g) { return g.rows >= 128 && g.Lk >= 64; }

// Enough row splits for the tiles of states to reach every SM, each of at least eight blocks of rows.
int cross_tc_backward_splits(const CrossGeom& g) {
    const int sms = sm_count(), tile_rows = g.d == 128 ? 128 : 256;
    const long long units = (long long)((g.Lk + tile_rows - 1) / tile_rows) * g.kv_heads * g.B;
    if (sms <= 0 || units <= 0 || units >= sms) return 1;
    long long s = sms / units;
    const long long most = ((g.rows + BN - 1) / BN) / 8;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

bra_status cross_backward_tc(const CrossGeom& g, int splits, const void* q, const void* k, const void* v,
                             const void* o, const float* lse, const void* grad_o, void* dq, void* dk, void* dv,
                             float* delta, float* parts, int* status, cudaStream_t stream) {
    return g.d == 32   ? launch_d<32>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, status, stream)
           : g.d == 64 ? launch_d<64>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, status, stream)
                       : launch_d<128>(g, splits, q, k, v, o, lse, grad_o, dq, dk, dv, delta, parts, status, stream);
}

}  // namespace bra
