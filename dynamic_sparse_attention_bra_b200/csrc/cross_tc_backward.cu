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
// S and dP have buffers for the blocks ahead (two at d = 128, three at d = 64:
// what the sums' 2 d columns leave), so that the products of the next block run
// under the exponentials of this one.  At d = 32 one buffer and two CTAs on an SM do
// the same, and hide the ends of short units as well (64 entries of 784 rows over 196
// states, 4 heads: 106 us for 125).  There is no maximum to agree on, so several
// threads share a row, in parts of 16 columns: four at d = 64; two, and at d = 128 two
// groups of such threads that take the blocks in turn, elsewhere.
// Roles of the warps: 0 issues S and dP, 1 the sums' products; 2 starts the loads
// (TMA, or cp.async where no map can be made); 3 passes each landed tile on, after
// it has zeroed the rows of masked or missing states (what is stored there must
// not reach a product) and, for dK and dV, added the columns' log sums and D; from
// 4 on the rows' threads.
// With two tiles of 128 rows a CTA, one buffer, and a thread a row (the first
// form) a block's products and exponentials took turns: 4250 clocks for two
// tiles, of which a row's threads waited 2360.
// Every mbarrier wait is bounded; on expiry the kernel records kDevTimeout, stops
// all roles, drains its products and frees TMEM.
#include "cross_map.h"
#include "cross_tc.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;

constexpr int kCtrl = 4;
constexpr int kParts = 4;   // 16-column parts of a block
constexpr int kStages = 4;  // at most
constexpr int BN = 64;      // columns of a block

struct Barriers {
    uint64_t c_land[kStages], c_full[kStages], c_empty[kStages];
    uint64_t r_land[2], r_full[2], r_empty[2];
    uint64_t s_full[3], p_full[3], acc_done[3];  // [buffer]
    uint64_t unit_done, rest_full, epi_done, drain[2];
    uint32_t words[kStages][2];  // dQ: the block's valid states
    uint32_t row_words[2][4];    // dK, dV: the tile's
    uint32_t tmem;
    int abort;
};

template <int D>
struct Cfg {
    static constexpr int kCtas = D == 32 ? 2 : 1;   // on an SM
    static constexpr int kBufs = D == 32 ? 1 : D == 64 ? 3 : 2;  // of S and dP
    static constexpr int kGroups = D == 128 ? 2 : 1;  // of row threads, taking blocks in turn
    static_assert(kBufs % kGroups == 0, "a group waits for every use of its buffers");
    static constexpr int kShare = D == 64 ? 4 : 2;    // threads of a row in a group
    static constexpr int kRowThreads = 128 * kGroups * kShare;
    static constexpr int kThreads = 32 * kCtrl + kRowThreads;
    // TMEM: buffer x: S at 128 x, dP at 128 x + 64 (P and dS over them); sums
    static constexpr uint32_t kCols = D == 32 ? 256 : 512;
    static constexpr uint32_t kDp = 64, kAcc1 = 128 * kBufs, kAcc2 = 128 * kBufs + D;
    static constexpr uint32_t kRow = 128u * D * 2u, kCol = (uint32_t)BN * D * 2u;
    static constexpr int kRing = D == 128 ? 3 : 4;
    // rows [buffer] x (R1 | R2), then stages of C1 | C2, the columns' statistics (dQ: a row's sums of dS), barriers
    static constexpr uint32_t kOffCol = 2 * 2 * kRow;
    static constexpr uint32_t kOffStat = kOffCol + kRing * 2 * kCol;
    static constexpr uint32_t kStat = kRing * 2 * BN * 4 > kRowThreads * 4 ? kRing * 2 * BN * 4 : kRowThreads * 4;
    static constexpr uint32_t kOffBar = kOffStat + kStat;
    static constexpr uint32_t kSmem = kOffBar + (uint32_t)sizeof(Barriers);  // (no room for an alignment's slack)
    static_assert(kSmem <= 227u * 1024u, "shared memory");
};

struct BwdPlan {
    int tiles;          // of 128 rows in a (entry, state head)
    int splits;         // dK, dV: parts of the rows of queries
    int units;
    int tma_r, tma_c;   // loads by TMA (the maps could be made)
};

struct Unit {
    int b, j, row0, split, n, t0, nb;  // first block and number of blocks
};

template <bool STATES>
__device__ __forceinline__ Unit unit_at(const CrossGeom& g, const BwdPlan& p, int u) {
    Unit x;
    x.row0 = (u % p.tiles) * 128;
    u /= p.tiles;
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

// STATES: the rows are states (dK, dV), the columns queries; else the rows are
// queries (dQ), the columns states.
template <int D, bool STATES>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
bra_cross_tc_backward_kernel(const __grid_constant__ CUtensorMap tr1, const __grid_constant__ CUtensorMap tr2,
                             const __grid_constant__ CUtensorMap tc1, const __grid_constant__ CUtensorMap tc2,
                             const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                             const __nv_bfloat16* o, const float* lse, const __nv_bfloat16* go, __nv_bfloat16* out1,
                             __nv_bfloat16* out2, float* delta, float* parts, CrossGeom g, BwdPlan p, int* status) {
    using C = Cfg<D>;
    constexpr int kRing = C::kRing, NB = C::kBufs, kShare = C::kShare, kGroups = C::kGroups;
    constexpr int kEach = kShare * kGroups;  // threads of a row
    constexpr int kPanels = D == 128 ? 2 : 1;  // of 64 channels (D = 32: one of 32)
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    if (sbase & 1023u) {  // the swizzled tiles need what the declaration asks for
        raise_status(status, kDevBounds);
        return;
    }
    Barriers* sb = reinterpret_cast<Barriers*>(smem + C::kOffBar);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(&sb->c_land[i], 1);
            ptx::mbar_init(&sb->c_full[i], 1);
            ptx::mbar_init(&sb->c_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(&sb->r_land[x], 1);
            ptx::mbar_init(&sb->r_full[x], 1);
            ptx::mbar_init(&sb->r_empty[x], STATES ? 1 : 1 + C::kRowThreads);  // the products; the reads of dO for D
            ptx::mbar_init(&sb->drain[x], 1);
        }
        for (int x = 0; x < NB; ++x) {
            ptx::mbar_init(&sb->s_full[x], 1);
            ptx::mbar_init(&sb->p_full[x], 128 * kShare);
            ptx::mbar_init(&sb->acc_done[x], 1);
        }
        ptx::mbar_init(&sb->unit_done, 1);
        ptx::mbar_init(&sb->rest_full, C::kRowThreads);
        ptx::mbar_init(&sb->epi_done, C::kRowThreads);
        sb->abort = 0;
        ptx::mbar_init_fence();
    }
    if (warp == 0) {
        ptx::tmem_alloc(&sb->tmem, C::kCols);
        ptx::tmem_relinquish();
        ptx::tc_fence_before();
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sb->tmem;
    grid_dependency_wait();

    auto col_tile = [&](int stage) { return sbase + C::kOffCol + (uint32_t)stage * 2u * C::kCol; };
    auto row_tile = [&](int use) { return sbase + (uint32_t)(use & 1) * 2u * C::kRow; };

    if (warp == 0) {
        // -------------------------------------------------------------- S and dP
        {
            int i = 0, use = 0;  // blocks and units so far
            bool ok = true;
            for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const Unit x = unit_at<STATES>(g, p, u);
                if (x.nb == 0) continue;
                ok = warp_wait(&sb->r_full[use & 1], (use >> 1) & 1, &sb->abort, status);
                const uint64_t r1 = k_major<D>(row_tile(use)), r2 = k_major<D>(row_tile(use) + C::kRow);
                for (int b = 0; ok && b < x.nb; ++b, ++i) {
                    const int stage = i % kRing, buf = i % NB;
                    const uint32_t cols = tmem + (uint32_t)buf * 128u;
                    const uint64_t c1 = k_major<D>(col_tile(stage)), c2 = k_major<D>(col_tile(stage) + C::kCol);
                    // the buffer holds the P and dS of two blocks ago until their products end
                    if (!warp_wait(&sb->c_full[stage], (i / kRing) & 1, &sb->abort, status) ||
                        (i >= NB && !warp_wait(&sb->acc_done[buf], (i / NB - 1) & 1, &sb->abort, status))) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t idesc = ptx::idesc_bf16_f32(128, block_cols<STATES>(x, b), false, false);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        ptx::warp_mma_bf16(cols, r1 + k_step<D>(kk, 128), c1 + k_step<D>(kk, BN), idesc, kk);
                        ptx::warp_mma_bf16(cols + C::kDp, r2 + k_step<D>(kk, 128), c2 + k_step<D>(kk, BN), idesc, kk);
                    }
                    ptx::warp_mma_commit(&sb->s_full[buf]);
                    if (b == x.nb - 1) ptx::warp_mma_commit(&sb->r_empty[use & 1]);
                }
                ++use;
            }
            ptx::warp_mma_commit(&sb->drain[0]);
            ptx::mbar_wait(&sb->drain[0], 0, kWait);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------- the sums
        {
            const uint32_t idesc = ptx::idesc_bf16_f32(128, D, false, true);
            int i = 0, use = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const Unit x = unit_at<STATES>(g, p, u);
                // the last unit's sums have been read
                if (x.nb > 0 && use++ > 0 && !warp_wait(&sb->epi_done, (use - 2) & 1, &sb->abort, status)) break;
                for (int b = 0; b < x.nb; ++b, ++i) {
                    const int stage = i % kRing, buf = i % NB;
                    const uint64_t c1 = n_major<D>(col_tile(stage), BN);
                    const uint64_t c2 = STATES ? n_major<D>(col_tile(stage) + C::kCol, BN) : c1;
                    const uint32_t cols = tmem + (uint32_t)buf * 128u;
                    if (!warp_wait(&sb->p_full[buf], (i / NB) & 1, &sb->abort, status)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const int steps = block_cols<STATES>(x, b) >> 4;
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        if (kk < steps) {
                            const uint32_t a = cols + (uint32_t)kk * 16u, more = kk > 0 ? 1u : (uint32_t)(b > 0);
                            ptx::warp_mma_bf16_ta(tmem + C::kAcc1, a + C::kDp, c1 + n_step<D>(kk), idesc, more);
                            ptx::warp_mma_bf16_ta(tmem + C::kAcc2, a, c2 + n_step<D>(kk), idesc, more);
                        }
                    ptx::warp_mma_commit(&sb->acc_done[buf]);
                    ptx::warp_mma_commit(&sb->c_empty[stage]);
                    if (b == x.nb - 1) ptx::warp_mma_commit(&sb->unit_done);
                }
            }
            ptx::warp_mma_commit(&sb->drain[1]);
            ptx::mbar_wait(&sb->drain[1], 0, kWait);
        }
        __syncwarp();
    } else if (warp == 2) {
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
            const Unit x = unit_at<STATES>(g, p, u);
            if (x.nb == 0) continue;
            // ``rows`` rows from r0 of both operands, states or queries, to dst and dst + second
            auto load = [&](uint32_t dst, uint32_t second, bool states, int r0, int rows, int tma, const CUtensorMap* m1,
                            const CUtensorMap* m2, uint64_t* land) {
                if (tma) {
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(land, 2u * (uint32_t)rows * D * 2u);
                        const int head = states ? x.j : x.j * g.rep, at = states ? r0 : r0 / g.rep;
                        const int b1 = (states ? g.k_batch : g.q_batch) ? x.b : 0, b2 = states && !g.v_batch ? 0 : x.b;
#pragma unroll
                        for (int c = 0; c < kPanels; ++c) {
                            ptx::tma_load_4d(dst + (uint32_t)(c * rows) * 128u, m1, c * 64, head, at, b1, land);
                            ptx::tma_load_4d(dst + second + (uint32_t)(c * rows) * 128u, m2, c * 64, head, at, b2, land);
                        }
                    }
                } else {
                    if (states) {
                        tc_load_states<D>(dst, k + (size_t)x.b * g.k_batch + (size_t)x.j * D, g.k_row, r0, x.n, rows, lane);
                        tc_load_states<D>(dst + second, v + (size_t)x.b * g.v_batch + (size_t)x.j * D, g.v_row, r0, x.n,
                                       rows, lane);
                    } else {
                        tc_load_queries<D>(dst, q, false, g, x.b, x.j, r0, rows, lane);
                        tc_load_queries<D>(dst + second, go, true, g, x.b, x.j, r0, rows, lane);
                    }
                    ptx::cp_async_wait_all();
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(land);
                }
            };
            uint32_t wr[4], w[2];
            if (STATES) valid_words(g, x.b, x.n, x.row0, lane, wr);
            if (use >= 2 && !warp_wait(&sb->r_empty[use & 1], ((use >> 1) - 1) & 1, &sb->abort, status)) break;
            if (STATES && lane == 0) {
#pragma unroll
                for (int h = 0; h < 4; ++h) sb->row_words[use & 1][h] = wr[h];
            }
            load(row_tile(use), C::kRow, STATES, x.row0, 128, p.tma_r, &tr1, &tr2, &sb->r_land[use & 1]);
            for (int b = 0; b < x.nb; ++b, ++i) {
                const int stage = i % kRing;
                if (!STATES) valid_words(g, x.b, x.n, (x.t0 + b) * BN, lane, w);
                if (i >= kRing && !warp_wait(&sb->c_empty[stage], ((i / kRing) - 1) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                if (!STATES && lane == 0) {
                    sb->words[stage][0] = w[0];
                    sb->words[stage][1] = w[1];
                }
                load(col_tile(stage), C::kCol, !STATES, (x.t0 + b) * BN, BN, p.tma_c, &tc1, &tc2, &sb->c_land[stage]);
            }
            ++use;
        }
    } else if (warp == 3) {
        // ------------------------------------------- landed tiles, passed to the products
        int i = 0, use = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<STATES>(g, p, u);
            if (x.nb == 0) continue;
            auto pass = [&](uint64_t* full) {  // this warp's stores, seen by the products and the rows' threads
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(full);
            };
            if (!warp_wait(&sb->r_land[use & 1], (use >> 1) & 1, &sb->abort, status)) break;
            if (STATES) clear_states<D, 4>(row_tile(use), C::kRow, sb->row_words[use & 1], lane);
            pass(&sb->r_full[use & 1]);
            float st[4];  // STATES: this lane's share of a block's log sums (2) and D (2), read a block ahead
            auto ahead = [&](int b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (x.t0 + b) * BN + h * 32 + lane;
                    const bool in = b < x.nb && r < g.rows;
                    const size_t at = in ? cross_lse_offset(g, x.b, x.j, r) : 0;
                    st[h] = in ? __ldcg(lse + at) : -INFINITY;
                    st[2 + h] = in ? __ldcg(delta + at) : 0.f;
                }
            };
            if (STATES) ahead(0);
            for (int b = 0; b < x.nb; ++b, ++i) {
                const int stage = i % kRing;
                if (!warp_wait(&sb->c_land[stage], (i / kRing) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                if constexpr (STATES) {
                    float* stat = reinterpret_cast<float*>(smem + C::kOffStat) + stage * 2 * BN;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        stat[h * 32 + lane] = -exponent_offset(st[h]);
                        stat[BN + h * 32 + lane] = -st[2 + h];
                    }
                } else {
                    clear_states<D, 2>(col_tile(stage), C::kCol, sb->words[stage], lane);
                }
                pass(&sb->c_full[stage]);
                if (STATES) ahead(b + 1);
            }
            ++use;
        }
    } else {
        // ---------------------------------------------------- P, dS and the epilogue
        // 16-column parts ``part``, + kShare .. of the group's blocks; ``mine`` of the row's threads
        const int mine = (warp - kCtrl) >> 2, part = mine % kShare, grp = mine / kShare, qd = warp & 3;
        const int row = 32 * qd + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * qd) << 16);
        const float c2 = g.scale * kLog2e;
        const uint64_t c22 = ptx::pack_f32x2(c2, c2);
        int i = 0, use = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<STATES>(g, p, u);
            const int r0 = x.row0 + row;
            const bool in = r0 < (STATES ? g.Lk : g.rows);
            float noff = -INFINITY, nd = 0.f;  // dQ: the row's -offset and -D0
            if (!STATES && x.nb > 0) {
                // D0 = <dO, O>: O from memory, dO from the tile
                float d0 = 0.f;
                const size_t off = in ? cross_o_offset(g, x.b, x.j, r0) : 0;
                uint4 ov[D / 8];
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    ov[c] = in ? __ldcg(reinterpret_cast<const uint4*>(o + off) + c) : make_uint4(0u, 0u, 0u, 0u);
                if (in) noff = -exponent_offset(__ldcg(lse + cross_lse_offset(g, x.b, x.j, r0)));
                if (!warp_wait(&sb->r_full[use & 1], (use >> 1) & 1, &sb->abort, status)) break;
                const uint8_t* r2 = smem + (size_t)(use & 1) * 2 * C::kRow + C::kRow;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    float a[8], h[8];
                    unpack16(ov[c], a, (const __nv_bfloat16*)nullptr);
                    unpack16(*reinterpret_cast<const uint4*>(r2 + op_offset<D>(row, c, 128)), h,
                             (const __nv_bfloat16*)nullptr);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d0 = fmaf(a[e], h[e], d0);
                }
                ptx::mbar_arrive(&sb->r_empty[use & 1]);
                nd = -d0;
            }
            uint64_t rest2 = 0ull;
            for (int b = 0; b < x.nb; ++b, ++i) {
                if (kGroups > 1 && i % kGroups != grp) continue;
                const int stage = i % kRing, buf = i % NB;
                const uint32_t cols = lanes + (uint32_t)buf * 128u;
                if (!warp_wait(&sb->s_full[buf], (i / NB) & 1, &sb->abort, status) ||
                    !warp_wait(&sb->c_full[stage], (i / kRing) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
#pragma unroll
                for (int pt = part; pt < kParts; pt += kShare) {
                    if (!STATES && block_cols<STATES>(x, b) <= pt * 16) break;
                    const float* stat = reinterpret_cast<const float*>(smem + C::kOffStat) + stage * 2 * BN + pt * 16;
                    uint32_t s[16], dp[16];
                    ptx::tmem_load_pair(cols + pt * 16, cols + C::kDp + pt * 16, s, dp);
                    const uint32_t w = STATES ? 0xffffu : (sb->words[stage][pt >> 1] >> ((pt & 1) * 16)) & 0xffffu;
                    uint32_t pp[8], pd[8];
                    auto form = [&](bool masked) {
                        const uint64_t noff2 = ptx::pack_f32x2(noff, noff), nd2 = ptx::pack_f32x2(nd, nd);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            uint64_t no = noff2, dd = nd2;
                            if constexpr (STATES) {
                                const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(stat + (e & ~1) * 2);
                                const ulonglong2 z = *reinterpret_cast<const ulonglong2*>(stat + BN + (e & ~1) * 2);
                                no = e & 1 ? a.y : a.x;
                                dd = e & 1 ? z.y : z.x;
                            }
                            float lo, hi, dlo, dhi;
                            ptx::unpack_f32x2(
                                ptx::fma_f32x2(ptx::pack_f32x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                                               c22, no),
                                lo, hi);
                            lo = ptx::ex2(lo);
                            hi = ptx::ex2(hi);
                            ptx::unpack_f32x2(
                                ptx::mul_f32x2(ptx::pack_f32x2(lo, hi),
                                               ptx::add_f32x2(ptx::pack_f32x2(__uint_as_float(dp[2 * e]),
                                                                              __uint_as_float(dp[2 * e + 1])),
                                                              dd)),
                                dlo, dhi);
                            if (masked) {  // nothing, whatever the columns hold
                                if (!((w >> (2 * e)) & 1u)) lo = dlo = 0.f;
                                if (!((w >> (2 * e + 1)) & 1u)) hi = dhi = 0.f;
                            }
                            pp[e] = ptx::pack_bf16x2(lo, hi);
                            pd[e] = ptx::pack_bf16x2(dlo, dhi);
                            // the sum of dS as it enters the product: taking it out of dQ takes the roundings' sum
                            // out too, which would multiply what K's states have in common
                            if (!STATES)
                                rest2 = ptx::add_f32x2(rest2, ptx::pack_f32x2(__uint_as_float(pd[e] << 16),
                                                                              __uint_as_float(pd[e] & 0xffff0000u)));
                        }
                    };
                    if (STATES || w == 0xffffu) form(false);
                    else form(true);
                    // over the first 8 of the 16 scores that this thread has read
                    ptx::tmem_st8(cols + pt * 16, pp);
                    ptx::tmem_st8(cols + C::kDp + pt * 16, pd);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&sb->p_full[buf]);
            }
            if (!ok) break;
            if (x.nb > 0) {
                // (a barrier of the units: a group that has not seen the last but one use of the last block's buffer
                // could not wait for the last by its parity)
                if (!warp_wait(&sb->unit_done, use & 1, &sb->abort, status)) break;
                ptx::tc_fence_after();
            }
            bool live = x.nb > 0;
            float rest = 0.f;  // dQ: D - D0
            size_t at = 0;
            if (STATES) {
                live = live && in && r0 < x.n && (!g.kv_mask || __ldcg(g.kv_mask + (size_t)x.b * g.Lk + r0) != 0);
                if (in) at = (((size_t)x.b * g.Lk + r0) * g.kv_heads + x.j) * D;
            } else {
                if (x.nb > 0) {
                    float lo, hi;
                    ptx::unpack_f32x2(rest2, lo, hi);
                    float* rests = reinterpret_cast<float*>(smem + C::kOffStat);
                    rests[mine * 128 + row] = lo + hi;
                    ptx::mbar_arrive(&sb->rest_full);
                    if (!warp_wait(&sb->rest_full, use & 1, &sb->abort, status)) break;
#pragma unroll
                    for (int y = 0; y < kEach; ++y) rest += rests[y * 128 + row];
                }
                if (in) {
                    at = cross_o_offset(g, x.b, x.j, r0);
                    if (mine == 0) delta[cross_lse_offset(g, x.b, x.j, r0)] = rest - nd;
                }
            }
            const size_t elems = (size_t)g.B * g.Lk * g.kv_heads * D;
#pragma unroll 1
            for (int c = mine * (D / kEach); c < (mine + 1) * (D / kEach); c += 8) {
                __syncwarp();  // rows past the last store nothing, but stay with their warp for its loads
                uint32_t a1[8], a2[8];
                if (x.nb > 0) ptx::tmem_load_pair(lanes + C::kAcc1 + c, lanes + C::kAcc2 + c, a1, a2);
                float f1[8], f2[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f1[e] = live ? __uint_as_float(a1[e]) : 0.f;
                    f2[e] = live ? __uint_as_float(a2[e]) : 0.f;
                    if (!STATES) f1[e] = fmaf(-rest, f2[e], f1[e]);
                    f1[e] *= g.scale;
                }
                if (STATES && in && p.splits > 1) {
                    float* out = parts + (size_t)x.split * 2 * elems + at + c;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        *reinterpret_cast<float4*>(out + e) = make_float4(f1[e], f1[e + 1], f1[e + 2], f1[e + 3]);
                        *reinterpret_cast<float4*>(out + elems + e) = make_float4(f2[e], f2[e + 1], f2[e + 2], f2[e + 3]);
                    }
                } else if (in) {
                    *reinterpret_cast<uint4*>(out1 + at + c) =
                        make_uint4(ptx::pack_bf16x2(f1[0], f1[1]), ptx::pack_bf16x2(f1[2], f1[3]),
                                   ptx::pack_bf16x2(f1[4], f1[5]), ptx::pack_bf16x2(f1[6], f1[7]));
                    if (STATES)
                        *reinterpret_cast<uint4*>(out2 + at + c) =
                            make_uint4(ptx::pack_bf16x2(f2[0], f2[1]), ptx::pack_bf16x2(f2[2], f2[3]),
                                       ptx::pack_bf16x2(f2[4], f2[5]), ptx::pack_bf16x2(f2[6], f2[7]));
                }
            }
            if (x.nb > 0) {
                ++use;
                ptx::tc_fence_before();  // the next unit's first products may overwrite the sums
                ptx::mbar_arrive(&sb->epi_done);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    allow_dependents();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::kCols);
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
    p.tiles = ((STATES ? g.Lk : g.rows) + 127) / 128;
    p.splits = STATES ? splits : 1;
    const long long units = (long long)p.tiles * p.splits * g.kv_heads * g.B;
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
    if (!allow_shared<bra_cross_tc_backward_kernel<D, STATES>>(C::kSmem)) return BRA_ERR_CUDA;
    const int most = sms * C::kCtas, grid = units < most ? (int)units : most;
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

// A full tile of rows, a full block of states, and enough work for the tiles of 128
// to fill the SMs or, at d >= 64, to stream long enough; below, the warps' form with
// tiles of 64 is ahead.  Forward and both gradients, its time and this form's, in us:
//   d = 32   2 x 1024 rows x 1024 states (2^21 scores)  45 / 59, 64 x 192 x 256 (3 M)  26 / 30,
//            64 x 512 x 128 (2^22)  32 / 28, 64 x 1024 x 256 (2^24)  80 / 59
//   d = 64   2 x 128 x 128  19 / 21, 2 x 512 x 256  31 / 29, 2 x 128 x 4096 (2^20)  108 / 69,
//            64 x 128 x 64 (2^19)  18 / 23, 64 x 128 x 128 (2^20)  22 / 23, 64 x 128 x 256  30 / 27
//   d = 128  2 x 128 x 64  26 / 32, 2 x 128 x 256  38 / 36, 64 x 128 x 64 (2^19)  29 / 34,
//            64 x 128 x 128 (2^20)  40 / 34
bool cross_tc_backward_covers(const CrossGeom& g) {
    if (g.rows < 128 || g.Lk < 64) return false;
    return g.d == 32 ? cross_scores(g) >= 1LL << 22 : g.Lk >= 256 || cross_scores(g) >= 1LL << 20;
}

// Enough row splits for the tiles of states to fill the SMs, each of at least eight blocks of rows.
int cross_tc_backward_splits(const CrossGeom& g) {
    const int slots = sm_count() * (g.d == 32 ? Cfg<32>::kCtas : 1);
    const long long units = (long long)((g.Lk + 127) / 128) * g.kv_heads * g.B;
    if (slots <= 0 || units <= 0 || units >= slots) return 1;
    long long s = slots / units;
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
