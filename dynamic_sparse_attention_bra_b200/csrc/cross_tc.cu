// Cross attention to an encoder's states, bf16, on tcgen05 tensor cores: the
// form for many rows (a map's tokens, a decoder's prompt).  The mathematics
// is that of cross_mma.cu.
//
// A unit of work is two tiles of 128 rows (four at d = 32) of one (entry, state
// head) and a range of the states, streamed in blocks of 64 (128 at d = 64) that
// its tiles share.  Per tile and block: S = Q K^T (M 128, N = the block) lands in
// TMEM; a softmax thread per row takes its scores into registers, writes P as bf16
// into TMEM, and O += P V (P the TMEM operand, N = d) accumulates in TMEM.  O is
// rescaled only where a row's maximum has grown by more than 2^8 since the last
// rescale (until then P may exceed 1: its relative rounding is the same, and l, in
// fp32, uses the same offset), so that the common block costs no pass over O.
//
// Roles of the warps, one CTA on an SM: 0, 1 issue the products of the even, odd
// tiles; 2 starts the loads of K and V, and of the tiles' Q (double-buffered), by TMA
// (cp.async where no map can be made); 3 passes each landed block on, after it has
// zeroed V's rows of masked or missing states, so that what is stored there never
// reaches a product; from 4 on, four warps for each tile, the softmax.  For d <= 64
// the next S is issued as soon as the scores are in registers, under the
// exponentials.  For d = 128 the columns do not suffice for a P of its own: P
// takes its S's, and S has two buffers, so that the next S is there before this
// softmax ends.
//
// d = 32: a block costs a tile's threads its waits and TMEM latencies besides the
// exponentials, so four tiles share an SM (2 x 16,384 rows of 2 heads over 4096
// states: 107 us for 132 with two tiles and blocks of 128).
//
// Bound by the exponentials (16 a clock and SM) for d = 32, where they would take 61
// of those 107 us, by them and the products for d = 128 (4 x 2048 tokens of 16 heads
// on 4, up to 2048 states each: 103 to 119 us by the power
// that a run gets, 52 to 60 % of a large product's rate).
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
constexpr int kStages = 4;  // at most
constexpr float kGrow = 8.f;  // powers of two a maximum may grow by before O is rescaled

struct Barriers {
    uint64_t kv_land[kStages], kv_full[kStages], kv_empty[kStages];
    uint64_t q_full[4][2], q_empty[4][2];
    // [tile][buffer of the block]
    uint64_t s_full[4][2], s_free[4][2], p_full[4][2], o_done[4][2];
    uint64_t drain[2];
    uint32_t words[kStages][4];  // the block's valid states
    uint32_t tmem;
    int abort;
};

template <int D>
struct Cfg {
    static constexpr int kTiles = D == 32 ? 4 : 2;      // of 128 rows in a unit
    static constexpr int kThreads = 32 * (kCtrl + 4 * kTiles);
    static constexpr int kBlock = D == 64 ? 128 : 64;   // states of a block
    static constexpr int kBufs = D == 128 ? 2 : 1;      // of S and P
    static constexpr bool kAlias = D == 128;            // P in its S's columns
    static constexpr uint32_t kCols = 512;
    static constexpr uint32_t kTileCols = kCols / kTiles;
    // buffer x: S at x * 64, P at kP + x * 64; O
    static constexpr uint32_t kP = kAlias ? 0 : kBlock, kO = kAlias ? 128 : kBlock + kBlock / 2;
    static constexpr uint32_t kQTile = 128u * D * 2u, kKvTile = (uint32_t)kBlock * D * 2u;
    static constexpr int kRing = D == 128 ? 3 : 4;  // stages that fit beside Q
    static constexpr uint32_t kOffKv = 2 * kTiles * kQTile;  // Q [tile][2], then stages of K | V
    static constexpr uint32_t kOffBar = kOffKv + (uint32_t)kRing * 2u * kKvTile;
    static constexpr uint32_t kSmem = kOffBar + (uint32_t)sizeof(Barriers) + 1024u;
    static_assert(kSmem <= 227u * 1024u, "shared memory");
};

struct TcPlan {
    int groups;   // units' rows in a (entry, state head)
    int splits;
    int units;
    int tma_q, tma_kv;  // loads by TMA (a map could be made)
};

struct Unit {
    int b, j, row0, split, n, t0, nb;  // first block and number of blocks
};

template <int BN, int ROWS>
__device__ __forceinline__ Unit unit_at(const CrossGeom& g, const TcPlan& p, int u) {
    Unit x;
    x.row0 = (u % p.groups) * ROWS;
    u /= p.groups;
    x.split = u % p.splits;
    u /= p.splits;
    x.j = u % g.kv_heads;
    x.b = u / g.kv_heads;
    x.n = cross_len(g, x.b);
    const int all = (x.n + BN - 1) / BN, per = (all + p.splits - 1) / p.splits;
    x.t0 = x.split * per;
    x.nb = max(0, min(all, x.t0 + per) - x.t0);
    return x;
}

// Columns of scores that block t has: its states, in steps of 16.
template <int BN>
__device__ __forceinline__ int block_cols(int n, int t) { return (min(BN, n - t * BN) + 15) & ~15; }

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
bra_cross_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                    const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                    CrossParts parts, CrossGeom g, TcPlan p, int* status) {
    using C = Cfg<D>;
    constexpr int kRing = C::kRing, BN = C::kBlock, NB = C::kBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    Barriers* sb = reinterpret_cast<Barriers*>(smem + C::kOffBar);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(&sb->kv_land[i], 1);
            ptx::mbar_init(&sb->kv_full[i], 1);
            ptx::mbar_init(&sb->kv_empty[i], C::kTiles);
        }
        for (int x = 0; x < C::kTiles; ++x) {
            for (int y = 0; y < 2; ++y) {
                ptx::mbar_init(&sb->q_full[x][y], 1);
                ptx::mbar_init(&sb->q_empty[x][y], 1);
                ptx::mbar_init(&sb->s_full[x][y], 1);
                ptx::mbar_init(&sb->s_free[x][y], 128);
                ptx::mbar_init(&sb->p_full[x][y], 128);
                ptx::mbar_init(&sb->o_done[x][y], 1);
            }
            if (x < 2) ptx::mbar_init(&sb->drain[x], 1);
        }
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

    if (warp < 2) {
        // ---------------------------------------- products of tiles ``warp``, warp + 2
        constexpr int kOwn = C::kTiles / 2;
        const uint32_t idesc_o = ptx::idesc_bf16_f32(128, D, false, true);
        int i = 0;                              // blocks so far
        int done[kOwn] = {}, use[kOwn] = {};    // of these, the tile's own; its units
        bool ok = true;
        // S = Q K^T of the unit's b-th block, the ``at``-th in all
        auto qk = [&](const Unit& x, int y, int b, int at) -> bool {
            const int tile = warp + 2 * y, c = done[y] + b, stage = at % kRing, buf = c % NB;
            const uint32_t cols = tmem + (uint32_t)tile * C::kTileCols;
            if (!warp_wait(&sb->kv_full[stage], (at / kRing) & 1, &sb->abort, status)) return false;
            // the buffer's last S: read, or (P shares its columns) used by its P V
            if (c >= NB && !warp_wait(C::kAlias ? &sb->o_done[tile][buf] : &sb->s_free[tile][buf], (c / NB - 1) & 1,
                                      &sb->abort, status))
                return false;
            ptx::tc_fence_after();
            const uint64_t qd = k_major<D>(sbase + (uint32_t)(tile * 2 + (use[y] & 1)) * C::kQTile);
            const uint64_t kd = k_major<D>(sbase + C::kOffKv + (uint32_t)stage * 2u * C::kKvTile);
            const uint32_t idesc = ptx::idesc_bf16_f32(128, block_cols<BN>(x.n, x.t0 + b), false, false);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                ptx::warp_mma_bf16(cols + (uint32_t)buf * 64u, qd + k_step<D>(kk, 128), kd + k_step<D>(kk, BN), idesc, kk);
            ptx::warp_mma_commit(&sb->s_full[tile][buf]);
            if (b == x.nb - 1) ptx::warp_mma_commit(&sb->q_empty[tile][use[y] & 1]);
            return true;
        };
        // O += P V
        auto pv = [&](const Unit& x, int y, int b, int at) -> bool {
            const int tile = warp + 2 * y, c = done[y] + b, stage = at % kRing, buf = c % NB;
            const uint32_t cols = tmem + (uint32_t)tile * C::kTileCols;
            if (!warp_wait(&sb->p_full[tile][buf], (c / NB) & 1, &sb->abort, status)) return false;
            ptx::tc_fence_after();
            const uint64_t vd = n_major<D>(sbase + C::kOffKv + (uint32_t)stage * 2u * C::kKvTile + C::kKvTile, BN);
            const int steps = block_cols<BN>(x.n, x.t0 + b) >> 4;
            const uint32_t pt = cols + C::kP + (uint32_t)buf * 64u;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                if (kk < steps)
                    ptx::warp_mma_bf16_ta(cols + C::kO, pt + (uint32_t)kk * 8u, vd + n_step<D>(kk), idesc_o,
                                          kk > 0 ? 1u : (uint32_t)(b > 0));
            ptx::warp_mma_commit(&sb->o_done[tile][buf]);
            ptx::warp_mma_commit(&sb->kv_empty[stage]);
            return true;
        };
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<BN, 128 * C::kTiles>(g, p, u);
            bool on[kOwn];  // the tile has rows
#pragma unroll
            for (int y = 0; y < kOwn; ++y) on[y] = x.row0 + (warp + 2 * y) * 128 < g.rows;
            for (int b = -1; ok && b < x.nb; ++b) {
#pragma unroll
                for (int y = 0; y < kOwn; ++y) {
                    if (!ok || !on[y] || b + 1 >= x.nb) continue;
                    if (b < 0) ok = warp_wait(&sb->q_full[warp + 2 * y][use[y] & 1], (use[y] >> 1) & 1, &sb->abort, status);
                    ok = ok && qk(x, y, b + 1, i + b + 1);
                }
                if (b < 0) continue;
#pragma unroll
                for (int y = 0; y < kOwn; ++y) {
                    if (!ok) continue;
                    if (on[y]) {
                        ok = pv(x, y, b, i + b);
                    } else {
                        ok = warp_wait(&sb->kv_full[(i + b) % kRing], ((i + b) / kRing) & 1, &sb->abort, status);
                        if (lane == 0) ptx::mbar_arrive(&sb->kv_empty[(i + b) % kRing]);
                    }
                }
            }
            i += x.nb;
#pragma unroll
            for (int y = 0; y < kOwn; ++y)
                if (on[y] && x.nb > 0) {
                    done[y] += x.nb;
                    ++use[y];
                }
        }
        ptx::warp_mma_commit(&sb->drain[warp]);
        ptx::mbar_wait(&sb->drain[warp], 0, kWait);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------------ loads
        constexpr int kPanels = D == 128 ? 2 : 1;  // of 64 channels (D = 32: one of 32)
        if (lane == 0) {
            ptx::tma_prefetch_desc(&tq);
            ptx::tma_prefetch_desc(&tk);
            ptx::tma_prefetch_desc(&tv);
        }
        int i = 0, uses[C::kTiles] = {};
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<BN, 128 * C::kTiles>(g, p, u);
            if (x.nb == 0) continue;
#pragma unroll
            for (int tile = 0; tile < C::kTiles; ++tile) {
                const int row0 = x.row0 + tile * 128;
                if (!ok || row0 >= g.rows) continue;
                const int use = uses[tile]++;
                uint64_t* full = &sb->q_full[tile][use & 1];
                if (use >= 2 && !warp_wait(&sb->q_empty[tile][use & 1], ((use >> 1) - 1) & 1, &sb->abort, status)) {
                    ok = false;
                    continue;
                }
                const uint32_t qt = sbase + (uint32_t)(tile * 2 + (use & 1)) * C::kQTile;
                if (p.tma_q) {
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(full, C::kQTile);
#pragma unroll
                        for (int c = 0; c < kPanels; ++c)
                            ptx::tma_load_4d(qt + (uint32_t)c * 128u * 128u, &tq, c * 64, x.j * g.rep, row0 / g.rep,
                                             g.q_batch ? x.b : 0, full);
                    }
                } else {
                    tc_load_queries<D>(qt, q, false, g, x.b, x.j, row0, 128, lane);
                    ptx::cp_async_wait_all();
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(full);
                }
            }
            const __nv_bfloat16* kbase = k + (size_t)x.b * g.k_batch + (size_t)x.j * D;
            const __nv_bfloat16* vbase = v + (size_t)x.b * g.v_batch + (size_t)x.j * D;
            for (int b = 0; ok && b < x.nb; ++b, ++i) {
                const int stage = i % kRing, key0 = (x.t0 + b) * BN;
                uint32_t w[BN / 32];
                valid_words(g, x.b, x.n, key0, lane, w);
                if (i >= kRing && !warp_wait(&sb->kv_empty[stage], ((i / kRing) - 1) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                const uint32_t kt = sbase + C::kOffKv + (uint32_t)stage * 2u * C::kKvTile;
                uint64_t* land = &sb->kv_land[stage];
                if (lane == 0) {
#pragma unroll
                    for (int h = 0; h < BN / 32; ++h) sb->words[stage][h] = w[h];
                }
                if (p.tma_kv) {
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(land, 2u * C::kKvTile);
#pragma unroll
                        for (int c = 0; c < kPanels; ++c) {
                            ptx::tma_load_4d(kt + (uint32_t)c * BN * 128u, &tk, c * 64, x.j, key0, g.k_batch ? x.b : 0,
                                             land);
                            ptx::tma_load_4d(kt + C::kKvTile + (uint32_t)c * BN * 128u, &tv, c * 64, x.j, key0,
                                             g.v_batch ? x.b : 0, land);
                        }
                    }
                } else {
                    tc_load_states<D>(kt, kbase, g.k_row, key0, x.n, BN, lane);
                    tc_load_states<D>(kt + C::kKvTile, vbase, g.v_row, key0, x.n, BN, lane);
                    ptx::cp_async_wait_all();
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(land);
                }
            }
        }
    } else if (warp == 3) {
        // ---------------------------------------- landed blocks, passed to the products
        int i = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<BN, 128 * C::kTiles>(g, p, u);
            for (int b = 0; b < x.nb; ++b, ++i) {
                const int stage = i % kRing;
                if (!warp_wait(&sb->kv_land[stage], (i / kRing) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                // K's rows need not be cleared: their scores are replaced, and no sum runs over them
                const uint32_t vt = sbase + C::kOffKv + (uint32_t)stage * 2u * C::kKvTile + C::kKvTile;
                clear_states<D, BN / 32, 1>(vt, 0u, sb->words[stage], lane);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sb->kv_full[stage]);
            }
        }
    } else {
        // ------------------------------------------------------ softmax + epilogue
        const int tile = (warp - kCtrl) >> 2, qd = warp & 3;
        const int row = 32 * qd + lane;
        const uint32_t cols = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)tile * C::kTileCols;
        const float sl = g.scale * kLog2e;
        const uint64_t sl2 = ptx::pack_f32x2(sl, sl);
        int i = 0, done = 0;  // blocks so far; this tile's own
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at<BN, 128 * C::kTiles>(g, p, u);
            if (x.row0 + tile * 128 >= g.rows) {
                i += x.nb;
                continue;
            }
            float m = -INFINITY;
            uint64_t l2 = 0ull;
            for (int b = 0; b < x.nb; ++b, ++i, ++done) {
                const int buf = done % NB, phase = done / NB;
                const uint32_t scol = cols + (uint32_t)buf * 64u;
                if (!warp_wait(&sb->s_full[tile][buf], phase & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                // the row's scores; columns that no product wrote are masked below
                const int nc = block_cols<BN>(x.n, x.t0 + b);
                uint32_t r[BN / 32][32];
                ptx::tmem_load(scol, r);
                if constexpr (!C::kAlias) {
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&sb->s_free[tile][buf]);
                }
                const int left = x.n - (x.t0 + b) * BN;
                if (g.kv_mask || left < BN) {
                    // (the block has been passed on; the wait makes its words visible)
                    if (!warp_wait(&sb->kv_full[i % kRing], (i / kRing) & 1, &sb->abort, status)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int h = 0; h < BN / 32; ++h) {
                        const uint32_t w = sb->words[i % kRing][h];
                        if (w != 0xffffffffu) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((w >> e) & 1u)) r[h][e] = 0xff800000u;  // -inf
                        }
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int h = 0; h < BN / 32; ++h)
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mx[(e >> 1) & 3] =
                            ptx::max3(mx[(e >> 1) & 3], __uint_as_float(r[h][e]), __uint_as_float(r[h][e + 1]));
                const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
                // P's buffer: its last P V is done
                if (done >= NB && !warp_wait(&sb->o_done[tile][buf], (phase - 1) & 1, &sb->abort, status)) {
                    ok = false;
                    break;
                }
                if (b == 0) {
                    m = mn;
                } else if (__any_sync(0xffffffffu, mn > m + kGrow)) {
                    // O stands still once the previous block's P V is done
                    if (!warp_wait(&sb->o_done[tile][(done - 1) % NB], ((done - 1) / NB) & 1, &sb->abort, status)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const float to = mn > m + kGrow ? mn : m;
                    const float alpha = to == -INFINITY ? 1.f : ptx::ex2(m - to);
                    m = to;
                    float lo, hi;
                    ptx::unpack_f32x2(l2, lo, hi);
                    l2 = ptx::pack_f32x2(lo * alpha, hi * alpha);
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t r[16];
                        ptx::tmem_ld16(cols + C::kO + c, r);
                        ptx::tmem_wait16(r);
#pragma unroll
                        for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                        ptx::tmem_st16(cols + C::kO + c, r);
                    }
                }
                ptx::tc_fence_after();
                const float mu = m == -INFINITY ? 0.f : m;  // no valid state yet
                const uint64_t neg = ptx::pack_f32x2(-mu, -mu);
                // P = 2^(s - m) of 16 columns, rounded once to bf16 for the product
                auto chunk = [&](const uint32_t* sc, uint32_t col) {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float lo, hi;
                        ptx::unpack_f32x2(ptx::fma_f32x2(ptx::pack_f32x2(__uint_as_float(sc[2 * e]),
                                                                         __uint_as_float(sc[2 * e + 1])),
                                                         sl2, neg),
                                          lo, hi);
                        lo = ptx::ex2(lo);
                        hi = ptx::ex2(hi);
                        l2 = ptx::add_f32x2(l2, ptx::pack_f32x2(lo, hi));
                        pk[e] = ptx::pack_bf16x2(lo, hi);
                    }
                    ptx::tmem_st8(cols + C::kP + (uint32_t)buf * 64u + col / 2, pk);
                };
                if (nc == BN) {  // without branches the exponentials of the chunks overlap
#pragma unroll
                    for (int h = 0; h < BN / 16; ++h) chunk(r[h >> 1] + (h & 1) * 16, h * 16);
                } else {
#pragma unroll
                    for (int h = 0; h < BN / 16; ++h)
                        if (nc > h * 16) chunk(r[h >> 1] + (h & 1) * 16, h * 16);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&sb->p_full[tile][buf]);
            }
            if (!ok) break;
            if (x.nb > 0) {
                if (!warp_wait(&sb->o_done[tile][(done - 1) % NB], ((done - 1) / NB) & 1, &sb->abort, status)) break;
                ptx::tc_fence_after();
            }
            float lo, hi;
            ptx::unpack_f32x2(l2, lo, hi);
            const float l = lo + hi;
            const int r0 = x.row0 + tile * 128 + row;
            const bool in = r0 < g.rows;
            const float inv = inverse_sum(l);
            const size_t part = ((size_t)(x.split * g.B + x.b) * g.kv_heads + x.j) * g.rows + r0;
            __nv_bfloat16* orow = in ? o + cross_o_offset(g, x.b, x.j, r0) : o;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                __syncwarp();  // rows past the last store nothing, but stay with their warp for its loads
                uint32_t r[16];
                if (x.nb > 0) {
                    ptx::tmem_ld16(cols + C::kO + c, r);
                    ptx::tmem_wait16(r);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = 0u;
                }
                if (in && p.splits > 1) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4*>(parts.o + part * D + c + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
                } else if (in) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = ptx::pack_bf16x2(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
                    *reinterpret_cast<uint4*>(orow + c) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(orow + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            if (in) {
                if (p.splits > 1) parts.ml[part] = make_float2(m, l);
                else if (lse) lse[cross_lse_offset(g, x.b, x.j, r0)] = log_sum(m, l);
            }
            ptx::tc_fence_before();  // O is read before the next tile's first P V, which p_full orders after this
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

template <int D>
bra_status launch_d(const CrossGeom& g, const TcPlan& plan, int grid, const void* q, const void* k, const void* v,
                    void* o, float* lse, CrossParts parts, int* status, cudaStream_t stream) {
    using C = Cfg<D>;
    if (!allow_shared<bra_cross_tc_kernel<D>>(C::kSmem)) return BRA_ERR_CUDA;
    TcPlan p = plan;
    CUtensorMap tq = {}, tk = {}, tv = {};
    // a Q tile is 128 / rep tokens; where rep does not divide it, and where a step is too long, cp.async
    p.tma_q = 128 % g.rep == 0 && encode_heads_map(&tq, q, g.B, g.Lq, g.heads, D, g.q_row, g.q_batch, 128 / g.rep, g.rep);
    p.tma_kv = g.Lk >= C::kBlock && encode_heads_map(&tk, k, g.B, g.Lk, g.kv_heads, D, g.k_row, g.k_batch, C::kBlock, 1) &&
               encode_heads_map(&tv, v, g.B, g.Lk, g.kv_heads, D, g.v_row, g.v_batch, C::kBlock, 1);
    const cudaError_t e = launch_after_previous(
        bra_cross_tc_kernel<D>, dim3(grid), dim3(C::kThreads), C::kSmem, stream, tq, tk, tv,
        static_cast<const __nv_bfloat16*>(q),
        static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(o),
        lse, parts, g, p, status);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace

// A full tile of rows, and enough work that a unit's start, end and waits are few of
// its blocks and that units of 256 rows (512 at d = 32) fill the SMs; below, the
// warps' form with its smaller units is ahead.  Its time and this form's, in us:
//   d = 32   2 x 4096 rows x 1024 states (2^23 scores)  13 / 17, x 4096 (2^25)  57 / 38
//   d = 64   16 x 256 rows x 512 (2^21)  13 / 15, 64 x 128 x 512 (2^22)  14 / 12,
//            16 x 1024 x 512 (2^23)  20 / 15
//   d = 128  16 x 256 x 320 (1.3 M)  11 / 13.5, 64 x 256 x 256 (2^22)  13.7 / 12.7,
//            64 x 256 x 512 (2^23)  32 / 17
bool cross_tc_covers(const CrossGeom& g) {
    return g.rows >= 128 && cross_scores(g) >= (g.d == 32 ? 1LL << 24 : 1LL << 22);
}

int cross_tc_rows(const CrossGeom& g) { return 128 * (g.d == 32 ? Cfg<32>::kTiles : Cfg<64>::kTiles); }

bra_status cross_forward_tc(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o,
                            float* lse, CrossParts parts, int* status, cudaStream_t stream) {
    TcPlan p = {};
    p.groups = (g.rows + cross_tc_rows(g) - 1) / cross_tc_rows(g);
    p.splits = splits;
    const long long units = (long long)p.groups * splits * g.kv_heads * g.B;
    if (units > 0x3fffffffLL) return BRA_ERR_UNSUPPORTED;
    p.units = (int)units;
    const int sms = sm_count();
    if (sms <= 0) return BRA_ERR_CUDA;
    const long long most = sms;
    const int grid = units < most ? (int)units : (int)most;
    return g.d == 32   ? launch_d<32>(g, p, grid, q, k, v, o, lse, parts, status, stream)
           : g.d == 64 ? launch_d<64>(g, p, grid, q, k, v, o, lse, parts, status, stream)
                       : launch_d<128>(g, p, grid, q, k, v, o, lse, parts, status, stream);
}

}  // namespace bra
