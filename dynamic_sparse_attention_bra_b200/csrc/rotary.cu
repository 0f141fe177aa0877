// Rotary positions with several axes (time, height, width) on Q and K.
// Pair i of a token turns by the angle pos[axis(i)] inv_freq[i]:
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin),
// the same for every head, so a thread forms the sines and cosines of a few
// pairs of a token, keeps them in registers and turns those pairs of all heads
// of Q and K.
//
// Angles of far positions do not fit fp32 (a position of 100000 leaves 2^-7 of a
// turn).  A frequency in turns is kept as a 64-bit fraction F; position x F modulo
// 2^64 is then the angle modulo a turn, whole turns wrapping away, at the cost of
// two integer multiply-adds and good to 2^-31 of a turn over all 32-bit positions:
// 2^-33 for F's last unit and 2^-32 for the half of the product that is cut off.
// Sine and cosine of the reduced angle are fp32.
//
// Bound by HBM (Q and K are read and written once, in 16-byte vectors) and, with
// few heads to share an angle, by the sines.  64 x 56 x 56 tokens, 2 + 2 heads of 32
// in bf16, 103 MB: 24.9 us (4.1 TB/s) with kHeads = 4 heads in flight, 26.5 with two,
// 29.0 with one; a table of a CTA's sines from angles in fp64 took 33 to 40 us.
#include "kernels.h"
#include "rotary.h"
#include "tma_host.h"

namespace bra {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 256;
constexpr int kHeads = 4;         // heads of a thread in flight

// x / d for x d < 2^32, by the multiplier floor(2^32 / d) + 1 (d > 1): a CTA's
// counts are small, and a division by a value known at launch would cost more
// than the rotation.
struct Divisor {
    uint32_t d, m;
};
__device__ __forceinline__ int divide(int x, Divisor v) { return v.d == 1 ? x : (int)__umulhi((uint32_t)x, v.m); }
Divisor divisor(int d) { return {(uint32_t)d, d > 1 ? (uint32_t)((1ull << 32) / (uint32_t)d + 1) : 0u}; }

// A unit of work: V channels that hold V / 2 pairs (interleaved), or V first
// halves and their V partners P channels on (split halves), or V channels
// past 2 P that are copied.
template <typename T, int V>
__device__ __forceinline__ uint4 narrow(const float (&f)[V]) {
    if constexpr (V == 4) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        return *reinterpret_cast<uint4*>(h);
    }
}

// A frequency (radians a position) as a fraction of a turn, times 2^64, within one
// unit: its 24-bit m times 1 / (2 pi) as a 128-bit fraction, of which the 64 bits below
// the point are taken where its exponent puts the point (the multiplication by stored
// bits of the constant of Payne and Hanek, "Radian reduction for trigonometric
// functions", 1983).  A negative frequency is the negated fraction of its magnitude;
// what is formed as 1 - |t| in fp64 would lose the bits that far positions need.
__device__ __forceinline__ uint64_t turns_of(float f) {
    const uint64_t hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;
    const uint32_t bits = __float_as_uint(f), field = bits >> 23 & 255u;
    const uint64_t m = field ? bits & 0x7fffffu | 0x800000u : bits & 0x7fffffu;
    const uint64_t low = m * lo, mid = m * hi, carry = __umul64hi(m, lo);
    const uint64_t w1 = mid + carry, w2 = __umul64hi(m, hi) + (w1 < mid ? 1u : 0u);
    // f = m 2^(field - 150), so that the point's bits of (w2, w1, low) start here
    const int s = 214 - (int)(field ? field : 1u), r = s & 63;
    if (s < 0 || s >= 192) return 0ull;  // (past the contract, or less than a unit)
    const uint64_t a = s < 64 ? low : s < 128 ? w1 : w2, b = s < 64 ? w1 : s < 128 ? w2 : 0ull;
    const uint64_t t = r ? a >> r | b << (64 - r) : a;
    return bits >> 31 ? 0ull - t : t;
}

// PAIRED: a unit is two vectors (split halves); else one (interleaved).
template <typename T, int V, bool PAIRED>
__global__ void __launch_bounds__(kThreads, 3)
bra_rotary_kernel(const T* q, const T* k, const int32_t* pos, const float* inv_freq, T* qo, T* ko, RotaryGeom g,
                  int tokens_per_cta, int units_turn, Divisor units) {
    using U = uint4;
    constexpr int A = PAIRED ? V : V / 2;  // pairs of a unit
    __shared__ uint64_t turns[kMaxPairs];
    // CTA = consecutive tokens of one entry
    const int b = blockIdx.y, l0 = blockIdx.x * tokens_per_cta, here = min(tokens_per_cta, g.L - l0);
    grid_dependency_wait();
    for (int i = threadIdx.x; i < g.P; i += kThreads) {
        const uint64_t f = turns_of(__ldcg(inv_freq + i));
        turns[i] = g.inverse ? 0ull - f : f;
    }
    __syncthreads();

    for (int item = threadIdx.x; item < here * (int)units.d; item += kThreads) {
        const int tk = here > 1 ? divide(item, units) : 0, x = item - tk * (int)units.d, l = l0 + tk;
        const bool turn = x < units_turn;
        const int c = PAIRED && !turn ? 2 * g.P + (x - units_turn) * V : x * V;
        const bool pair = PAIRED && turn;
        const T* src[2] = {q + (size_t)b * g.q_batch + (size_t)l * g.q_row + c,
                           k + (size_t)b * g.k_batch + (size_t)l * g.k_row + c};
        T* dst[2] = {qo + (size_t)b * g.qo_batch + (size_t)l * g.qo_row + c,
                     ko + (size_t)b * g.ko_batch + (size_t)l * g.ko_row + c};
        U va[kHeads], vz[kHeads];
        // heads h .. h + kHeads - 1 of Q and then K
        auto fetch = [&](int h) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int y = h + i;
                if (y >= g.heads + g.kv_heads) break;
                const T* s = y < g.heads ? src[0] + y * g.d : src[1] + (y - g.heads) * g.d;
                va[i] = *reinterpret_cast<const U*>(s);
                if (pair) vz[i] = *reinterpret_cast<const U*>(s + g.P);
            }
        };
        fetch(0);
        float cs[A], sn[A];
        if (turn) {
            int p0, p1, p2;
            if (pos) {
                const int32_t* at = pos + (size_t)b * g.pos_batch + (size_t)l * 3;
                p0 = __ldcg(at);
                p1 = __ldcg(at + 1);
                p2 = __ldcg(at + 2);
            } else {
                const int row = l / g.W;
                p0 = row / g.H;
                p1 = row - p0 * g.H;
                p2 = l - row * g.W;
            }
#pragma unroll
            for (int e = 0; e < A; ++e) {
                const int i = PAIRED ? c + e : c / 2 + e;
                if (i >= g.P) break;  // (interleaved: the last unit may hold channels past the pairs)
                const int p = i < g.axis1 ? p0 : (i < g.axis2 ? p1 : p2);
                // the product's upper half, a signed fraction of a turn
                const int angle = (int)(((uint64_t)(int64_t)p * turns[i]) >> 32);
                sincospif((float)angle * 4.656612873077393e-10f, &sn[e], &cs[e]);  // 2^-31: half turns
            }
        }
        for (int h = 0; h < g.heads + g.kv_heads; h += kHeads) {
            if (h > 0) fetch(h);
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int y = h + i;
                if (y >= g.heads + g.kv_heads) break;
                T* d = y < g.heads ? dst[0] + y * g.d : dst[1] + (y - g.heads) * g.d;
                if (!turn) {
                    *reinterpret_cast<U*>(d) = va[i];
                } else if constexpr (PAIRED) {
                    float f[V], z[V];
                    unpack16(va[i], f, static_cast<const T*>(nullptr));
                    unpack16(vz[i], z, static_cast<const T*>(nullptr));
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float w = f[e] * cs[e] - z[e] * sn[e];
                        z[e] = z[e] * cs[e] + f[e] * sn[e];
                        f[e] = w;
                    }
                    *reinterpret_cast<U*>(d) = narrow<T, V>(f);
                    *reinterpret_cast<U*>(d + g.P) = narrow<T, V>(z);
                } else {
                    float f[V];
                    unpack16(va[i], f, static_cast<const T*>(nullptr));
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        if ((c + e) / 2 >= g.P) break;
                        const float w = f[e] * cs[e / 2] - f[e + 1] * sn[e / 2];
                        f[e + 1] = f[e + 1] * cs[e / 2] + f[e] * sn[e / 2];
                        f[e] = w;
                    }
                    *reinterpret_cast<U*>(d) = narrow<T, V>(f);
                }
            }
        }
    }
    allow_dependents();
}

// Split halves of which P channels are no whole vectors: a pair's channels lie at
// different places of two vectors.  A thread has one vector of a token in all heads;
// the rows go through shared memory, where it reads its channels' partners, and the
// CTA's sines are a table there.  (64 x 56 x 56 tokens, 2 + 2 heads of 32 in bf16, 15
// pairs: 44 us; two-byte loads and stores of whole pairs 57.)
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 4)
bra_rotary_split_kernel(const T* q, const T* k, const int32_t* pos, const float* inv_freq, T* qo, T* ko, RotaryGeom g,
                        int tokens_per_cta, int tokens_per_pass, Divisor units, Divisor pairs) {
    __shared__ uint64_t turns[kMaxPairs];
    __shared__ float2 table[kThreads * V / 2];  // (cosine, sine) [token][pair]
    __shared__ __align__(16) T rows[kThreads * kHeads * V];  // [token][head][channel]
    const int b = blockIdx.y, l0 = blockIdx.x * tokens_per_cta, l1 = min(l0 + tokens_per_cta, g.L);
    const int tk = divide(threadIdx.x, units), c = ((int)threadIdx.x - tk * (int)units.d) * V;
    const int all = g.heads + g.kv_heads;
    grid_dependency_wait();
    for (int i = threadIdx.x; i < g.P; i += kThreads) {
        const uint64_t f = turns_of(__ldcg(inv_freq + i));
        turns[i] = g.inverse ? 0ull - f : f;
    }
    for (int first = l0; first < l1; first += tokens_per_pass) {
        const int here = min(tokens_per_pass, l1 - first), l = first + tk;
        const bool in = tk < here;
        const size_t in_q = (size_t)b * g.q_batch + (size_t)l * g.q_row + c, in_k = (size_t)b * g.k_batch + (size_t)l * g.k_row + c;
        const size_t out_q = (size_t)b * g.qo_batch + (size_t)l * g.qo_row + c,
                     out_k = (size_t)b * g.ko_batch + (size_t)l * g.ko_row + c;
        uint4 va[kHeads];
        auto fetch = [&](int h) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int y = h + i;
                if (in && y < all)
                    va[i] = *reinterpret_cast<const uint4*>(y < g.heads ? q + in_q + y * g.d : k + in_k + (y - g.heads) * g.d);
            }
        };
        fetch(0);
        __syncthreads();  // the frequencies are there; the last pass's table and rows are read
        for (int e = threadIdx.x; e < here * g.P; e += kThreads) {
            const int t = divide(e, pairs), i = e - t * g.P, at = first + t;
            int p;
            if (pos) {
                p = __ldcg(pos + (size_t)b * g.pos_batch + (size_t)at * 3 + (i < g.axis1 ? 0 : (i < g.axis2 ? 1 : 2)));
            } else {
                const int row = at / g.W, time = row / g.H;
                p = i < g.axis1 ? time : (i < g.axis2 ? row - time * g.H : at - row * g.W);
            }
            const int angle = (int)(((uint64_t)(int64_t)p * turns[i]) >> 32);
            float2 v;
            sincospif((float)angle * 4.656612873077393e-10f, &v.y, &v.x);
            table[e] = v;
        }
        float2 turn[V];  // (cosine, +- sine) of this thread's channels
        for (int h = 0; h < all; h += kHeads) {
            if (h > 0) {
                fetch(h);
                __syncthreads();  // the last heads' rows are read
            }
            T* mine = rows + (size_t)tk * kHeads * g.d + c;
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (in && h + i < all) *reinterpret_cast<uint4*>(mine + i * g.d) = va[i];
            __syncthreads();
            if (!in) continue;
            if (h == 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int j = c + e;
                    turn[e] = j >= 2 * g.P ? make_float2(1.f, 0.f) : table[tk * g.P + (j < g.P ? j : j - g.P)];
                    if (j < g.P) turn[e].y = -turn[e].y;
                }
            }
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int y = h + i;
                if (y >= all) break;
                float f[V], z[V];
                unpack16(va[i], f, static_cast<const T*>(nullptr));
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int j = c + e;
                    z[e] = to_f32(mine[i * g.d + e + (j < g.P ? g.P : j < 2 * g.P ? -g.P : 0)]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (c + e < 2 * g.P) f[e] = f[e] * turn[e].x + z[e] * turn[e].y;
                *reinterpret_cast<uint4*>(y < g.heads ? qo + out_q + y * g.d : ko + out_k + (y - g.heads) * g.d) =
                    narrow<T, V>(f);
            }
        }
    }
    allow_dependents();
}

template <typename T, int V>
cudaError_t launch_split(const RotaryGeom& g, const void* q, const void* k, const int32_t* pos, const float* inv_freq,
                         void* q_out, void* k_out, cudaStream_t stream) {
    const int units = g.d / V, pass = kThreads / units;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // two passes a CTA where that still gives each SM four CTAs
    const int per = (long long)g.B * g.L * units > 8LL * kThreads * sms ? 2 * pass : pass;
    return launch_after_previous(bra_rotary_split_kernel<T, V>, dim3((unsigned)((g.L + per - 1) / per), (unsigned)g.B),
                                 dim3(kThreads), 0, stream, static_cast<const T*>(q), static_cast<const T*>(k), pos,
                                 inv_freq, static_cast<T*>(q_out), static_cast<T*>(k_out), g, per, pass,
                                 divisor(units), divisor(g.P));
}

template <typename T, int V, bool PAIRED>
cudaError_t launch(const RotaryGeom& g, const void* q, const void* k, const int32_t* pos, const float* inv_freq,
                   void* q_out, void* k_out, cudaStream_t stream) {
    const int units_turn = PAIRED ? g.P / V : (2 * g.P + V - 1) / V;
    const int units = PAIRED ? units_turn + (g.d - 2 * g.P) / V : g.d / V;
    // a unit a thread and pass; two passes where that still gives each SM four CTAs
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const long long items = (long long)g.B * g.L * units;
    int per = (items > 8LL * kThreads * sms ? 2 : 1) * kThreads / units;
    if (per > g.L) per = g.L;
    if (per < 1) per = 1;
    return launch_after_previous(bra_rotary_kernel<T, V, PAIRED>, dim3((unsigned)((g.L + per - 1) / per), (unsigned)g.B),
                                 dim3(kThreads), 0, stream, static_cast<const T*>(q), static_cast<const T*>(k), pos,
                                 inv_freq, static_cast<T*>(q_out), static_cast<T*>(k_out), g, per, units_turn,
                                 divisor(units));
}

}  // namespace

bra_status rotary_launch(const RotaryGeom& g, bool bf16, const void* q, const void* k, const int32_t* pos,
                         const float* inv_freq, void* q_out, void* k_out, cudaStream_t stream) {
    const int v = bf16 ? 8 : 4;
    cudaError_t e;
    // split halves whose P channels are whole vectors pair them in a thread's registers
    const bool wide = g.P % v == 0;
    if (g.interleaved)
        e = bf16 ? launch<__nv_bfloat16, 8, false>(g, q, k, pos, inv_freq, q_out, k_out, stream)
                 : launch<float, 4, false>(g, q, k, pos, inv_freq, q_out, k_out, stream);
    else if (wide)
        e = bf16 ? launch<__nv_bfloat16, 8, true>(g, q, k, pos, inv_freq, q_out, k_out, stream)
                 : launch<float, 4, true>(g, q, k, pos, inv_freq, q_out, k_out, stream);
    else
        e = bf16 ? launch_split<__nv_bfloat16, 8>(g, q, k, pos, inv_freq, q_out, k_out, stream)
                 : launch_split<float, 4>(g, q, k, pos, inv_freq, q_out, k_out, stream);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace bra
