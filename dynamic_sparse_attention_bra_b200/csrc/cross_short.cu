// Cross attention to few states (at most 256), bf16, d = 32 or 64, on warp-level
// tensor-core products: the form for a map's tokens that read a short text or a
// small map.  The mathematics is that of cross_mma.cu.
//
// All valid states of a (entry, state head) fit in shared memory beside a few
// others', so a CTA loads them once and its warps then work on their own, each
// on tiles of 16 rows, with no synchronisation until the CTA's rows reach the next
// (entry, state head).  The tiles of the whole call are dealt to the CTAs in equal
// consecutive shares.
//
// Q goes from memory to the products' registers without shared memory: a
// thread of a quad takes 16-byte chunks t, t + 4 of a row, whatever channels the
// fragment layout names, and K's fragments take the same order (a dot product
// does not mind), as one 16-byte shared load for two products.  The next tile's Q
// is loaded under this tile's products; O leaves in 16-byte stores after a 4 x 4
// exchange in the quad.
// Bound by the latency of a warp's chain (about 550 instructions for 16 rows and 64
// states, half of the issue slots) and the first loads: 200,704 x 2 rows over 77 states
// (lengths from 39 on) take 32 us, of which
// memory would take 8; the tcgen05 form takes 51-61 us there, its roles' hand-over
// costing more than the work of one short block.
#include "cross_tile.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace bra {
namespace {

using namespace cross;
using wmma16::mma16816;
using wmma16::mma16816_first;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxStates = 256;
constexpr int kCtas = 2;  // on an SM (three of 80 registers a thread: 34.7 us for 31.7)

// K is read as 16-byte chunks by quads: at 128-byte rows, odd rows swap their halves.
template <int D>
__device__ __forceinline__ uint32_t k_offset(int r, int c) {
    return D == 32 ? (uint32_t)(r * 64 + c * 16) : (uint32_t)(r * 128 + ((c ^ ((r & 1) << 2)) << 4));
}

// w[i] of the four threads of a quad, thread t's w[i] becoming thread i's w[t].
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t) {
    const bool odd = t & 1, high = t & 2;
    uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), b = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
    if (odd) {
        w[0] = a;
        w[2] = b;
    } else {
        w[1] = a;
        w[3] = b;
    }
    a = __shfl_xor_sync(0xffffffffu, high ? w[0] : w[2], 2);
    b = __shfl_xor_sync(0xffffffffu, high ? w[1] : w[3], 2);
    if (high) {
        w[0] = a;
        w[1] = b;
    } else {
        w[2] = a;
        w[3] = b;
    }
}

// One warp's tile of 16 rows: its Q, running maxima and sums, and O.
template <int D>
struct Tile {
    uint4 q[2][D / 32];  // rows gq, gq + 8
    float acc[D / 8][4], mx[2], sum[2];
};

// 16 STEPS states from the tiles at k_lane (this thread's chunks) and sv, words
// their validity.  FIRST: the tile's first states.
template <int D, int STEPS, bool FIRST>
__device__ __forceinline__ void attend(Tile<D>& x, uint32_t k_lane, uint32_t k_next, uint32_t sv, const uint32_t* words,
                                       float sl, int lane) {
    const int t4 = lane & 3;
    float s[2 * STEPS][4];
#pragma unroll
    for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
        for (int m = 0; m < D / 32; ++m) {
            uint4 kv;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(kv.x), "=r"(kv.y), "=r"(kv.z), "=r"(kv.w)
                         : "r"(k_lane + (uint32_t)(i * 8 * D * 2) + (m ? k_next : 0u)));
            if (m == 0) mma16816_first(s[i], x.q[0][m].x, x.q[1][m].x, x.q[0][m].y, x.q[1][m].y, kv.x, kv.y);
            else mma16816(s[i], x.q[0][m].x, x.q[1][m].x, x.q[0][m].y, x.q[1][m].y, kv.x, kv.y);
            mma16816(s[i], x.q[0][m].z, x.q[1][m].z, x.q[0][m].w, x.q[1][m].w, kv.z, kv.w);
        }
#pragma unroll
    for (int i = 0; i < 2 * STEPS; i += 4) {
        const uint32_t w = words[i >> 2];
        if (w != 0xffffffffu) {
#pragma unroll
            for (int y = i; y < i + 4 && y < 2 * STEPS; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (!((w >> ((y - i) * 8 + t4 * 2 + e)) & 1u)) s[y][e] = s[y][2 + e] = -INFINITY;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float mn = fmaxf(s[0][2 * h], s[0][2 * h + 1]);
#pragma unroll
        for (int i = 1; i < 2 * STEPS; ++i) mn = ptx::max3(mn, s[i][2 * h], s[i][2 * h + 1]);
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2)) * sl;
        if (!FIRST) {
            mn = fmaxf(mn, x.mx[h]);
            const float f = ptx::ex2(x.mx[h] - (mn == -INFINITY ? 0.f : mn));
            x.sum[h] *= f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                x.acc[i][2 * h] *= f;
                x.acc[i][2 * h + 1] *= f;
            }
        } else {
            x.sum[h] = 0.f;
        }
        x.mx[h] = mn;
    }
    const float n0 = x.mx[0] == -INFINITY ? 0.f : -x.mx[0], n1 = x.mx[1] == -INFINITY ? 0.f : -x.mx[1];
    const uint64_t sl2 = ptx::pack_f32x2(sl, sl), n02 = ptx::pack_f32x2(n0, n0), n12 = ptx::pack_f32x2(n1, n1);
    uint64_t sums[2] = {ptx::pack_f32x2(x.sum[0], 0.f), ptx::pack_f32x2(x.sum[1], 0.f)};
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        uint32_t pa[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {  // tile 2 i + y / 2, row gq or gq + 8
            const float* sc = s[2 * i + (y >> 1)] + 2 * (y & 1);
            float lo, hi;
            ptx::unpack_f32x2(ptx::fma_f32x2(ptx::pack_f32x2(sc[0], sc[1]), sl2, y & 1 ? n12 : n02), lo, hi);
            lo = ptx::ex2(lo);
            hi = ptx::ex2(hi);
            sums[y & 1] = ptx::add_f32x2(sums[y & 1], ptx::pack_f32x2(lo, hi));
            pa[y] = ptx::pack_bf16x2(lo, hi);
        }
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
            uint32_t bf[4];
            frag_nn<D>(sv + (uint32_t)(i * 16 * D * 2), 0, c, lane, bf);
            if (FIRST && i == 0) {
                mma16816_first(x.acc[c], pa[0], pa[1], pa[2], pa[3], bf[0], bf[1]);
                mma16816_first(x.acc[c + 1], pa[0], pa[1], pa[2], pa[3], bf[2], bf[3]);
            } else {
                mma16816(x.acc[c], pa[0], pa[1], pa[2], pa[3], bf[0], bf[1]);
                mma16816(x.acc[c + 1], pa[0], pa[1], pa[2], pa[3], bf[2], bf[3]);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float lo, hi;
        ptx::unpack_f32x2(sums[h], lo, hi);
        x.sum[h] = lo + hi;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtas)
bra_cross_short_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                       const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                       CrossGeom g, int row_tiles, long long tiles, int pad) {
    constexpr int M = D / 32;  // 16-byte chunks of a row that a thread holds
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t words[kMaxStates / 32];
    const uint32_t sk = ptx::smem_addr(smem), sv = sk + (uint32_t)pad * D * 2u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t4 = lane & 3;
    const float sl = g.scale * kLog2e;
    const size_t q_step = (size_t)(g.q_row / 8), o_step = (size_t)g.heads * (D / 8);
    grid_dependency_wait();

    long long at = tiles * blockIdx.x / gridDim.x;
    const long long end = tiles * (blockIdx.x + 1) / gridDim.x;
    while (at < end) {
        const int item = (int)(at / row_tiles), first = (int)(at - (long long)item * row_tiles);
        const int last = (int)min((long long)row_tiles, first + (end - at));
        const int j = item % g.kv_heads, b = item / g.kv_heads;
        at += last - first;
        const int n = cross_len(g, b), n16 = (n + 15) & ~15;

        // steps between rows of Q and O in 16 bytes: rows of one token are consecutive heads
        const uint4* qb = reinterpret_cast<const uint4*>(q + (size_t)b * g.q_batch + (size_t)j * g.rep * D) + t4;
        uint4* ob = reinterpret_cast<uint4*>(o + ((size_t)b * g.Lq * g.heads + (size_t)j * g.rep) * D) + t4;
        uint4 qn[2][M];  // rows gq, gq + 8 of the warp's next tile
        auto fetch = [&](int tile) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = tile * 16 + h * 8 + gq;
                const bool on = tile < last && r < g.rows;
                int t = r, hh = 0;
                if (g.rep > 1) {
                    t = r / g.rep;
                    hh = r - t * g.rep;
                }
                const uint4* src = qb + (size_t)(uint32_t)t * q_step + hh * (D / 8);
#pragma unroll
                for (int m = 0; m < M; ++m) qn[h][m] = on ? __ldcg(src + 4 * m) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        fetch(first + warp);

        __syncthreads();  // the last item's states are read
        if (warp == 0) {
            for (int h = 0; h < kMaxStates / 32; ++h) {
                const int key = h * 32 + lane;
                const bool on = key < n && (!g.kv_mask || __ldcg(g.kv_mask + (size_t)b * g.Lk + key) != 0);
                const uint32_t w = __ballot_sync(0xffffffffu, on);
                if (lane == 0) words[h] = w;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < n16 * (D / 8); e += kThreads) {
            const int r = e / (D / 8), c = e % (D / 8);
            const bool on = (words[r >> 5] >> (r & 31)) & 1u;
            ptx::cp_async16_zfill(sk + k_offset<D>(r, c),
                                  on ? k + (size_t)b * g.k_batch + (size_t)r * g.k_row + j * D + c * 8 : k, on ? 16u : 0u);
            ptx::cp_async16_zfill(sv + tile_offset<D>(r, c),
                                  on ? v + (size_t)b * g.v_batch + (size_t)r * g.v_row + j * D + c * 8 : v, on ? 16u : 0u);
        }
        ptx::cp_async_wait_all();
        __syncthreads();

        for (int tile = first + warp; tile < last; tile += kWarps) {
            Tile<D> x;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int m = 0; m < M; ++m) x.q[h][m] = qn[h][m];
                x.mx[h] = -INFINITY;
                x.sum[h] = 0.f;
            }
            fetch(tile + kWarps);
            // this thread's chunks of the first eight states' rows (the swizzle repeats every two rows)
            const uint32_t k_lane = sk + k_offset<D>(gq, t4), k_next = k_offset<D>(gq, t4 + 4) - k_offset<D>(gq, t4);
            // straight code for every number of 16-state steps: guards and a loop between them cost as much again
            switch (min(n16, 64) >> 4) {
                case 0:
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x.acc[i][e] = 0.f;
                    break;
                case 1: attend<D, 1, true>(x, k_lane, k_next, sv, words, sl, lane); break;
                case 2: attend<D, 2, true>(x, k_lane, k_next, sv, words, sl, lane); break;
                case 3: attend<D, 3, true>(x, k_lane, k_next, sv, words, sl, lane); break;
                default: attend<D, 4, true>(x, k_lane, k_next, sv, words, sl, lane); break;
            }
            for (int c0 = 64; c0 < n16; c0 += 64) {
                const uint32_t kc = k_lane + (uint32_t)(c0 * D * 2), vc = sv + (uint32_t)(c0 * D * 2);
                const uint32_t* wc = words + (c0 >> 5);
                switch (min(n16 - c0, 64) >> 4) {
                    case 1: attend<D, 1, false>(x, kc, k_next, vc, wc, sl, lane); break;
                    case 2: attend<D, 2, false>(x, kc, k_next, vc, wc, sl, lane); break;
                    case 3: attend<D, 3, false>(x, kc, k_next, vc, wc, sl, lane); break;
                    default: attend<D, 4, false>(x, kc, k_next, vc, wc, sl, lane); break;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x.sum[h] += __shfl_xor_sync(0xffffffffu, x.sum[h], 1);
                x.sum[h] += __shfl_xor_sync(0xffffffffu, x.sum[h], 2);
                const int r = tile * 16 + h * 8 + gq;
                const float inv = inverse_sum(x.sum[h]);
                int t = r, hh = 0;
                if (g.rep > 1) {
                    t = r / g.rep;
                    hh = r - t * g.rep;
                }
                uint4* dst = ob + (size_t)(uint32_t)t * o_step + hh * (D / 8);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = ptx::pack_bf16x2(x.acc[4 * m + i][2 * h] * inv, x.acc[4 * m + i][2 * h + 1] * inv);
                    quad_transpose(w, t4);
                    if (r < g.rows) dst[4 * m] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (lse && t4 == 0 && r < g.rows)
                    lse[((size_t)b * g.heads + (size_t)(j * g.rep + hh)) * g.Lq + t] = log_sum(x.mx[h], x.sum[h]);
            }
        }
    }
    allow_dependents();
}

template <int D>
bra_status launch_d(const CrossGeom& g, const void* q, const void* k, const void* v, void* o, float* lse,
                    cudaStream_t stream) {
    const int pad = (g.Lk + 15) & ~15, row_tiles = (g.rows + 15) / 16;
    const uint32_t bytes = (uint32_t)(pad > 0 ? pad : 16) * D * 4u;
    const long long tiles = (long long)row_tiles * g.kv_heads * g.B;
    const int sms = sm_count();
    if (sms <= 0) return BRA_ERR_CUDA;
    if (!allow_shared<bra_cross_short_kernel<D>>(kMaxStates * D * 4)) return BRA_ERR_CUDA;
    // CTAs that keep to one (entry, state head), a tile a warp, where those fit on the
    // SMs at once (32 entries of 32 rows over 64 states: 4 us; equal shares, which cross
    // from one to the next and load twice, 11 us), else two an SM with equal shares
    const long long most = (long long)kCtas * sms;
    const long long whole = (long long)g.kv_heads * g.B * ((row_tiles + kWarps - 1) / kWarps);
    const int grid = (int)(whole < most ? whole : most);
    const cudaError_t e = launch_after_previous(
        bra_cross_short_kernel<D>, dim3(grid), dim3(kThreads), bytes, stream, static_cast<const __nv_bfloat16*>(q),
        static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(o), lse,
        g, row_tiles, tiles, pad);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace

// At d = 64 a small call is left to the streaming form, whose first tile of states is
// there sooner (2 x 1024 rows over 256 states: 7.2 us for 8.9), a large one with more
// than two of tcgen05's blocks to it (128 x 1024 rows over 192 states: 31 us for 34,
// over 256: 33 for 43; over 128 both take 26).
bool cross_short_covers(const CrossGeom& g) {
    if (g.rows <= 16 || g.Lk > kMaxStates || g.d > 64) return false;
    if (g.d == 32) return true;
    const double scores = cross_scores(g);
    return scores >= 1LL << 19 && (g.Lk <= 128 || scores < 1LL << 23);
}

bra_status cross_forward_short(const CrossGeom& g, const void* q, const void* k, const void* v, void* o, float* lse,
                               cudaStream_t stream) {
    return g.d == 32 ? launch_d<32>(g, q, k, v, o, lse, stream) : launch_d<64>(g, q, k, v, o, lse, stream);
}

}  // namespace bra
