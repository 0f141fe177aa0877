// Cross attention to an encoder's states, bf16, on tcgen05 tensor cores: the
// form for many rows (a map's tokens, a decoder's prompt).  The mathematics
// is that of cross_mma.cu.
//
// A unit of work is 256 rows of one (entry, state head), two tiles of 128, and
// a range of the states, streamed in blocks of 64 that both tiles share.  Per
// tile and block: S = Q K^T (M 128, N up to 64) lands in TMEM; a softmax
// thread per row reads its scores twice (maximum, then exponentials), writes P
// as bf16 into TMEM, and O += P V (P the TMEM operand, N = d) accumulates in
// TMEM.  O is rescaled only where a row's maximum has grown by more than 2^8
// since the last rescale (until then P may exceed 1: its relative rounding
// is the same, and l, in fp32, uses the same offset), so that the common
// block costs no pass over O.
//
// Roles of the 12 warps: 0, 1 issue the products of tile 0, 1; 2, 3 load (16-byte
// cp.async, masked or missing rows filled with zeros: blocks of the states in turn,
// and the tile's Q, double-buffered); 4-7, 8-11 are the tiles' softmax.  Two
// such CTAs run on an SM for d <= 64 (256 TMEM columns each), one for d = 128.
// For d = 64 P takes S's columns, and the next S waits for P V; otherwise P has
// columns of its own, and the next S is issued before P V.
//
// Bound by the exponentials (16 a clock and SM) for d = 32, by them and the
// products for d = 128.  Every mbarrier wait is bounded; on expiry the kernel
// records kDevTimeout, stops all roles, drains its products and frees TMEM.
#include "cross_tile.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;

constexpr int kCtrl = 4;
constexpr int kThreads = 32 * (kCtrl + 8);
constexpr int kStages = 4;
constexpr uint32_t kWait = 1u << 22;
constexpr float kGrow = 8.f;  // powers of two a maximum may grow by before O is rescaled

struct Barriers {
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t q_full[2][2], q_empty[2][2];
    uint64_t s_full[2], s_free[2], p_full[2], o_done[2], drain[2];
    uint32_t words[kStages][2];  // the block's valid states
    uint32_t tmem;
    int abort;
};

template <int D>
struct Cfg {
    static constexpr bool kAlias = D == 64;
    static constexpr int kCtas = D <= 64 ? 2 : 1;
    static constexpr uint32_t kCols = D <= 64 ? 256 : 512;
    static constexpr uint32_t kGroupCols = kCols / 2;
    static constexpr uint32_t kP = kAlias ? 0 : 64, kO = kAlias ? 64 : 96;
    static constexpr uint32_t kQTile = 128u * D * 2u, kKvTile = 64u * D * 2u;
    static constexpr int kRing = D == 32 ? 4 : D == 64 ? 2 : 3;  // stages that fit beside Q
    static constexpr uint32_t kOffKv = 4 * kQTile;        // Q [group][2], then stages of K | V
    static constexpr uint32_t kOffBar = kOffKv + (uint32_t)kRing * 2u * kKvTile;
    static constexpr uint32_t kSmem = kOffBar + (uint32_t)sizeof(Barriers) + 1024u;
};

// Byte offset of 16-byte chunk c of row r in a tile of ``rows`` rows: 64-byte
// rows with the 64-byte swizzle at D = 32; 128-byte rows with the 128-byte
// swizzle otherwise, channels 64.. of D = 128 in a second panel.
template <int D>
__device__ __forceinline__ uint32_t op_offset(int r, int c, int rows) {
    if constexpr (D == 32) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Descriptor of a K-major operand (rows x D) at its k-th 16 channels.
template <int D>
__device__ __forceinline__ uint64_t k_major(uint32_t tile, int kk, int rows) {
    if constexpr (D == 32) return ptx::smem_desc(tile + kk * 32, 16, 512, ptx::kSwizzle64B);
    return ptx::smem_desc(tile + (uint32_t)((kk >> 2) * rows * 128 + (kk & 3) * 32), 16, 1024, ptx::kSwizzle128B);
}
// Descriptor of V (64 states x D, channels the N axis) at its k-th 16 states.
template <int D>
__device__ __forceinline__ uint64_t v_operand(uint32_t tile, int kk) {
    if constexpr (D == 32) return ptx::smem_desc(tile + kk * 1024, 16, 512, ptx::kSwizzle64B);
    return ptx::smem_desc(tile + kk * 2048, 64 * 128, 1024, ptx::kSwizzle128B);
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Barriers* sb, int* status) {
    for (uint32_t i = 0; i < kWait; ++i) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((i & 1023) == 1023 && *reinterpret_cast<volatile int*>(&sb->abort) != 0) return false;
    }
    *reinterpret_cast<volatile int*>(&sb->abort) = 1;
    raise_status(status, kDevTimeout);
    return false;
}

// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Barriers* sb, int* status) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, sb, status));
}

struct TcPlan {
    int pairs;    // units of 256 rows in a (entry, state head)
    int splits;
    int units;
};

struct Unit {
    int b, j, row0, split, n, t0, nb;  // first block and number of blocks
};

__device__ __forceinline__ Unit unit_at(const CrossGeom& g, const TcPlan& p, int u) {
    Unit x;
    x.row0 = (u % p.pairs) * 256;
    u /= p.pairs;
    x.split = u % p.splits;
    u /= p.splits;
    x.j = u % g.kv_heads;
    x.b = u / g.kv_heads;
    x.n = cross_len(g, x.b);
    const int all = (x.n + 63) / 64, per = (all + p.splits - 1) / p.splits;
    x.t0 = x.split * per;
    x.nb = max(0, min(all, x.t0 + per) - x.t0);
    return x;
}

// Columns of scores that block t has: its states, in steps of 16.
__device__ __forceinline__ int block_cols(int n, int t) { return (min(64, n - t * 64) + 15) & ~15; }

template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtas)
bra_cross_tc_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                    const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                    CrossParts parts, CrossGeom g, TcPlan p, int* status) {
    using C = Cfg<D>;
    constexpr int kRing = C::kRing;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    Barriers* sb = reinterpret_cast<Barriers*>(smem + C::kOffBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(&sb->kv_full[i], 32);
            ptx::mbar_init(&sb->kv_empty[i], 2);
        }
        for (int x = 0; x < 2; ++x) {
            for (int y = 0; y < 2; ++y) {
                ptx::mbar_init(&sb->q_full[x][y], 32);
                ptx::mbar_init(&sb->q_empty[x][y], 1);
            }
            ptx::mbar_init(&sb->s_full[x], 1);
            ptx::mbar_init(&sb->s_free[x], 128);
            ptx::mbar_init(&sb->p_full[x], 128);
            ptx::mbar_init(&sb->o_done[x], 1);
            ptx::mbar_init(&sb->drain[x], 1);
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
        // ------------------------------------------------ products of tile ``warp``
        if (lane == 0) {
            const int grp = warp;
            const uint32_t cols = tmem + (uint32_t)grp * C::kGroupCols;
            const uint32_t idesc_o = ptx::idesc_bf16_f32(128, D, false, true);
            int kb = 0, use = 0;  // blocks and tiles so far
            bool ok = true;
            auto pv = [&](const Unit& x, int b, int kk0) -> bool {  // O += P V of block b, the tile's kk0-th in all
                const int stage = kk0 % kRing;
                if (!wait_or_abort(&sb->p_full[grp], kk0 & 1, sb, status)) return false;
                ptx::tc_fence_after();
                const uint32_t vt = sbase + C::kOffKv + (uint32_t)stage * 2u * C::kKvTile + C::kKvTile;
                const int steps = block_cols(x.n, x.t0 + b) >> 4;
                for (int kk = 0; kk < steps; ++kk)
                    ptx::mma_bf16_ta(cols + C::kO, cols + C::kP + (uint32_t)kk * 8u, v_operand<D>(vt, kk), idesc_o,
                                     b > 0 || kk > 0);
                ptx::mma_commit(&sb->o_done[grp]);
                ptx::mma_commit(&sb->kv_empty[stage]);
                return true;
            };
            for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const Unit x = unit_at(g, p, u);
                if (x.nb == 0) continue;
                ok = wait_or_abort(&sb->q_full[grp][use & 1], (use >> 1) & 1, sb, status);
                const uint32_t qt = sbase + (uint32_t)(grp * 2 + (use & 1)) * C::kQTile;
                for (int b = 0; ok && b < x.nb; ++b) {
                    const int i = kb + b, stage = i % kRing;
                    if (!wait_or_abort(&sb->kv_full[stage], (i / kRing) & 1, sb, status) ||
                        (i > 0 && !wait_or_abort(C::kAlias ? &sb->o_done[grp] : &sb->s_free[grp], (i - 1) & 1, sb,
                                                 status))) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t kt = sbase + C::kOffKv + (uint32_t)stage * 2u * C::kKvTile;
                    const uint32_t idesc = ptx::idesc_bf16_f32(128, block_cols(x.n, x.t0 + b), false, false);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        ptx::mma_bf16(cols, k_major<D>(qt, kk, 128), k_major<D>(kt, kk, 64), idesc, kk);
                    ptx::mma_commit(&sb->s_full[grp]);
                    if (b == x.nb - 1) ptx::mma_commit(&sb->q_empty[grp][use & 1]);
                    if constexpr (C::kAlias) {
                        ok = pv(x, b, i);
                    } else {
                        if (b > 0) ok = pv(x, b - 1, i - 1);
                    }
                }
                if (!C::kAlias && ok) ok = pv(x, x.nb - 1, kb + x.nb - 1);
                kb += x.nb;
                ++use;
            }
            ptx::mma_commit(&sb->drain[grp]);
            ptx::mbar_wait(&sb->drain[grp], 0, kWait);
        }
        __syncwarp();
    } else if (warp < kCtrl) {
        // ------------------------------------------------------------------ loads
        const int grp = warp - 2;
        int kb = 0, use = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at(g, p, u);
            if (x.nb == 0) continue;
            if (use >= 2 && !warp_wait(&sb->q_empty[grp][use & 1], ((use >> 1) - 1) & 1, sb, status)) break;
            {
                const uint32_t qt = sbase + (uint32_t)(grp * 2 + (use & 1)) * C::kQTile;
                const int row0 = x.row0 + grp * 128;
#pragma unroll 4
                for (int e = lane; e < 128 * (D / 8); e += 32) {
                    const int r = e / (D / 8), c = e % (D / 8);
                    const bool on = row0 + r < g.rows;
                    ptx::cp_async16_zfill(qt + op_offset<D>(r, c, 128),
                                          on ? q + cross_q_offset(g, x.b, x.j, row0 + r) + c * 8 : q, on ? 16u : 0u);
                }
                ptx::cp_async_wait_all();
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&sb->q_full[grp][use & 1]);
            }
            const __nv_bfloat16* kbase = k + (size_t)x.b * g.k_batch + (size_t)x.j * D;
            const __nv_bfloat16* vbase = v + (size_t)x.b * g.v_batch + (size_t)x.j * D;
            for (int b = 0; b < x.nb; ++b) {
                const int i = kb + b, stage = i % kRing;
                if ((i & 1) != grp) continue;  // the other loader's block
                const int key0 = (x.t0 + b) * 64;
                uint32_t w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = key0 + h * 32 + lane;
                    w[h] = __ballot_sync(0xffffffffu,
                                         key < x.n && (!g.kv_mask || __ldcg(g.kv_mask + (size_t)x.b * g.Lk + key) != 0));
                }
                if (i >= kRing && !warp_wait(&sb->kv_empty[stage], ((i / kRing) - 1) & 1, sb, status)) {
                    ok = false;
                    break;
                }
                const uint32_t kt = sbase + C::kOffKv + (uint32_t)stage * 2u * C::kKvTile;
#pragma unroll 4
                for (int e = lane; e < 64 * (D / 8); e += 32) {
                    const int r = e / (D / 8), c = e % (D / 8);
                    const bool on = ((r < 32 ? w[0] : w[1]) >> (r & 31)) & 1u;
                    const uint32_t at = op_offset<D>(r, c, 64);
                    ptx::cp_async16_zfill(kt + at, on ? kbase + (size_t)(key0 + r) * g.k_row + c * 8 : k, on ? 16u : 0u);
                    ptx::cp_async16_zfill(kt + C::kKvTile + at, on ? vbase + (size_t)(key0 + r) * g.v_row + c * 8 : v,
                                          on ? 16u : 0u);
                }
                if (lane == 0) {
                    sb->words[stage][0] = w[0];
                    sb->words[stage][1] = w[1];
                }
                ptx::cp_async_wait_all();
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&sb->kv_full[stage]);
            }
            kb += x.nb;
            ++use;
        }
    } else {
        // ------------------------------------------------------ softmax + epilogue
        const int grp = (warp - kCtrl) >> 2, qd = warp & 3;
        const int row = 32 * qd + lane;
        const uint32_t cols = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)grp * C::kGroupCols;
        const float sl = g.scale * kLog2e;
        const uint64_t sl2 = ptx::pack_f32x2(sl, sl);
        int i = 0;  // blocks so far
        bool ok = true;
        for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
            const Unit x = unit_at(g, p, u);
            float m = -INFINITY;
            uint64_t l2 = 0ull;
            for (int b = 0; b < x.nb; ++b, ++i) {
                const int stage = i % kRing;
                if (!warp_wait(&sb->kv_full[stage], (i / kRing) & 1, sb, status) ||
                    !warp_wait(&sb->s_full[grp], i & 1, sb, status)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t w0 = sb->words[stage][0], w1 = sb->words[stage][1];
                const int nc = block_cols(x.n, x.t0 + b);
                const bool whole = (w0 & w1) == 0xffffffffu;
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    if (c >= nc) break;
                    uint32_t r[2][16];
                    ptx::tmem_ld16(cols + c, r[0]);
                    ptx::tmem_ld16(cols + c + 16, r[1]);
                    ptx::tmem_wait16(r[0]);
                    ptx::tmem_wait16(r[1]);
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            mx[e & 1] = fmaxf(mx[e & 1], fmaxf(__uint_as_float(r[0][e]), __uint_as_float(r[1][e])));
                    } else {
                        const uint32_t w = c == 0 ? w0 : w1;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if ((w >> e) & 1u) mx[e & 1] = fmaxf(mx[e & 1], __uint_as_float(r[e >> 4][e & 15]));
                    }
                }
                const float mn = fmaxf(mx[0], mx[1]) * sl;
                // the previous block's P V: its P is overwritten below, its O may be rescaled
                if (i > 0 && !warp_wait(&sb->o_done[grp], (i - 1) & 1, sb, status)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                if (b == 0) {
                    m = mn;
                } else if (__any_sync(0xffffffffu, mn > m + kGrow)) {
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
                const float mu = m == -INFINITY ? 0.f : m;  // no valid state yet
                const uint64_t neg = ptx::pack_f32x2(-mu, -mu);
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    if (c >= nc) break;
                    uint32_t r[16], pk[8];
                    ptx::tmem_ld16(cols + c, r);
                    ptx::tmem_wait16(r);
                    if (!whole) {
                        const uint32_t w = (c < 32 ? w0 : w1) >> (c & 31);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (!((w >> e) & 1u)) r[e] = 0xff800000u;  // -inf
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float lo, hi;
                        ptx::unpack_f32x2(ptx::fma_f32x2(ptx::pack_f32x2(__uint_as_float(r[2 * e]),
                                                                         __uint_as_float(r[2 * e + 1])),
                                                         sl2, neg),
                                          lo, hi);
                        lo = ptx::ex2(lo);
                        hi = ptx::ex2(hi);
                        l2 = ptx::add_f32x2(l2, ptx::pack_f32x2(lo, hi));
                        pk[e] = ptx::pack_bf16x2(lo, hi);
                    }
                    // d = 64: P overwrites scores that this thread has read (chunks 0.. of S hold P's chunks 0..)
                    ptx::tmem_st8(cols + C::kP + c / 2, pk);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                if constexpr (!C::kAlias) ptx::mbar_arrive(&sb->s_free[grp]);
                ptx::mbar_arrive(&sb->p_full[grp]);
            }
            if (!ok) break;
            if (x.nb > 0) {
                if (!warp_wait(&sb->o_done[grp], (i - 1) & 1, sb, status)) break;
                ptx::tc_fence_after();
            }
            float lo, hi;
            ptx::unpack_f32x2(l2, lo, hi);
            const float l = lo + hi;
            const int r0 = x.row0 + grp * 128 + row;
            const bool in = r0 < g.rows;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const size_t part = ((size_t)(x.split * g.B + x.b) * g.kv_heads + x.j) * g.rows + r0;
            __nv_bfloat16* orow = in ? o + cross_o_offset(g, x.b, x.j, r0) : o;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t r[16];
                if (x.nb > 0) {
                    ptx::tmem_ld16(cols + C::kO + c, r);
                    ptx::tmem_wait16(r);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = 0u;
                }
                if (!in) continue;
                if (p.splits > 1) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4*>(parts.o + part * D + c + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
                } else {
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
                else if (lse) lse[cross_lse_offset(g, x.b, x.j, r0)] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
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
bra_status launch_d(const CrossGeom& g, const TcPlan& p, int grid, const void* q, const void* k, const void* v,
                    void* o, float* lse, CrossParts parts, int* status, cudaStream_t stream) {
    using C = Cfg<D>;
    if (cudaFuncSetAttribute(bra_cross_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) !=
        cudaSuccess)
        return BRA_ERR_CUDA;
    const cudaError_t e = launch_after_previous(
        bra_cross_tc_kernel<D>, dim3(grid), dim3(kThreads), C::kSmem, stream, static_cast<const __nv_bfloat16*>(q),
        static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(o),
        lse, parts, g, p, status);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace

bool cross_tc_covers(const CrossGeom& g) { return g.rows >= 128; }

int cross_tc_rows() { return 256; }

bra_status cross_forward_tc(const CrossGeom& g, int splits, const void* q, const void* k, const void* v, void* o,
                            float* lse, CrossParts parts, int* status, cudaStream_t stream) {
    TcPlan p;
    p.pairs = (g.rows + 255) / 256;
    p.splits = splits;
    const long long units = (long long)p.pairs * splits * g.kv_heads * g.B;
    if (units > 0x3fffffffLL) return BRA_ERR_UNSUPPORTED;
    p.units = (int)units;
    const int sms = sm_count();
    if (sms <= 0) return BRA_ERR_CUDA;
    const long long most = (long long)sms * (g.d <= 64 ? 2 : 1);
    const int grid = units < most ? (int)units : (int)most;
    return g.d == 32   ? launch_d<32>(g, p, grid, q, k, v, o, lse, parts, status, stream)
           : g.d == 64 ? launch_d<64>(g, p, grid, q, k, v, o, lse, parts, status, stream)
                       : launch_d<128>(g, p, grid, q, k, v, o, lse, parts, status, stream);
}

}  // namespace bra
