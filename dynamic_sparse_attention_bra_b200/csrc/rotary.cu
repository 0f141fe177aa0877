// Rotary positions with several axes (time, height, width) on Q and K.
// Pair i of a token turns by the angle pos[axis(i)] inv_freq[i]:
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin),
// the same for every head, so a CTA forms the sines and cosines of its tokens
// once, in shared memory, and applies them to all heads of Q and K.
//
// Angles of far positions do not fit fp32 (a position of 100000 leaves 2^-7
// of a turn), so position x frequency and its reduction to a fraction of a
// turn are done in fp64; sine and cosine of the reduced angle in fp32.
//
// Bound by HBM: Q and K are read and written once, in 16-byte vectors, four
// units a thread, whose loads are issued before the CTA's angles are formed, so
// that forming them runs under the loads (ROTARY_NOTE).
#include "kernels.h"
#include "rotary.h"
#include "tma_host.h"

namespace bra {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 2048;  // (token, pair) angles of a CTA: 16 KB of shared memory
constexpr int kUnits = 4;         // units of a thread
constexpr int kMaxTokens = 256;   // of a CTA

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
struct Vec {
    using type = uint4;
};
template <>
struct Vec<__nv_bfloat16, 1> {
    using type = __nv_bfloat16;
};
template <>
struct Vec<float, 1> {
    using type = float;
};

template <typename T, int V>
__device__ __forceinline__ void widen(const typename Vec<T, V>::type& x, float (&f)[V]) {
    if constexpr (V == 1) f[0] = to_f32(x);
    else unpack16(x, f, static_cast<const T*>(nullptr));
}
template <typename T, int V>
__device__ __forceinline__ typename Vec<T, V>::type narrow(const float (&f)[V]) {
    if constexpr (V == 1) {
        return from_f32<T>(f[0]);
    } else if constexpr (V == 4) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        uint4 u;
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u = *reinterpret_cast<uint4*>(h);
        return u;
    }
}

// PAIRED: a unit is two vectors (split halves); else one (interleaved).
template <typename T, int V, bool PAIRED>
__global__ void __launch_bounds__(kThreads)
bra_rotary_kernel(const T* q, const T* k, const int32_t* pos, const float* inv_freq, T* qo, T* ko, RotaryGeom g,
                  int tokens_per_cta, int units_turn, Divisor per_token, Divisor per_head, Divisor pairs) {
    using U = typename Vec<T, V>::type;
    __shared__ float2 table[kMaxAngles];
    __shared__ int place[kMaxTokens][3];
    // CTA = consecutive tokens of one entry
    const int b = blockIdx.y, l0 = blockIdx.x * tokens_per_cta, here = min(tokens_per_cta, g.L - l0);
    const int units = here * (int)per_token.d;
    grid_dependency_wait();

    // the unit's channels c (and P + c), where they come from and go to
    struct Unit {
        const T* src;
        T* dst;
        int tab, c;  // first angle of the token; first channel, or -1
        bool turn;
        U a, z;
    } un[kUnits];
    auto fetch = [&](int u0) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = u0 + i * kThreads;
            un[i].c = -1;
            if (u >= units) continue;
            const int tk = here > 1 ? divide(u, per_token) : 0, w = u - tk * (int)per_token.d;
            const int head = divide(w, per_head), x = w - head * (int)per_head.d, l = l0 + tk;
            if (head < g.heads) {
                un[i].src = q + (size_t)b * g.q_batch + (size_t)l * g.q_row + (size_t)head * g.d;
                un[i].dst = qo + (size_t)b * g.qo_batch + (size_t)l * g.qo_row + (size_t)head * g.d;
            } else {
                un[i].src = k + (size_t)b * g.k_batch + (size_t)l * g.k_row + (size_t)(head - g.heads) * g.d;
                un[i].dst = ko + (size_t)b * g.ko_batch + (size_t)l * g.ko_row + (size_t)(head - g.heads) * g.d;
            }
            un[i].tab = tk * g.P;
            un[i].turn = x < units_turn;
            un[i].c = PAIRED && !un[i].turn ? 2 * g.P + (x - units_turn) * V : x * V;
            un[i].a = *reinterpret_cast<const U*>(un[i].src + un[i].c);
            if (PAIRED && un[i].turn) un[i].z = *reinterpret_cast<const U*>(un[i].src + g.P + un[i].c);
        }
    };
    fetch(threadIdx.x);

    for (int tk = threadIdx.x; tk < here; tk += kThreads) {
        const int l = l0 + tk;
        if (pos) {
#pragma unroll
            for (int axis = 0; axis < 3; ++axis)
                place[tk][axis] = __ldcg(pos + (size_t)b * g.pos_batch + (size_t)l * 3 + axis);
        } else {
            const int row = l / g.W, t = row / g.H;
            place[tk][0] = t;
            place[tk][1] = row - t * g.H;
            place[tk][2] = l - row * g.W;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < here * g.P; e += kThreads) {
        const int tk = divide(e, pairs), i = e - tk * g.P;
        const int p = place[tk][i < g.axis1 ? 0 : (i < g.axis2 ? 1 : 2)];
        // turns, reduced to [-1/2, 1/2]
        double turns = (double)p * (double)__ldcg(inv_freq + i) * 0.15915494309189533577;
        turns -= rint(turns);
        float s, c;
        sincospif(2.f * (float)turns, &s, &c);
        table[e] = make_float2(c, g.inverse ? -s : s);
    }
    __syncthreads();

    for (int u0 = threadIdx.x; u0 < units; u0 += kUnits * kThreads) {
        if (u0 != (int)threadIdx.x) fetch(u0);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int c = un[i].c;
            if (c < 0) continue;
            const float2* tab = table + un[i].tab;
            if (!un[i].turn) {
                *reinterpret_cast<U*>(un[i].dst + c) = un[i].a;
            } else if constexpr (PAIRED) {
                float f[V], h[V];
                widen<T, V>(un[i].a, f);
                widen<T, V>(un[i].z, h);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 t = tab[c + e];
                    const float y = f[e] * t.x - h[e] * t.y;
                    h[e] = h[e] * t.x + f[e] * t.y;
                    f[e] = y;
                }
                *reinterpret_cast<U*>(un[i].dst + c) = narrow<T, V>(f);
                *reinterpret_cast<U*>(un[i].dst + g.P + c) = narrow<T, V>(h);
            } else {
                float f[V];
                widen<T, V>(un[i].a, f);
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    if ((c + e) / 2 >= g.P) continue;  // the last unit may hold channels past the pairs
                    const float2 t = tab[(c + e) / 2];
                    const float y = f[e] * t.x - f[e + 1] * t.y;
                    f[e + 1] = f[e + 1] * t.x + f[e] * t.y;
                    f[e] = y;
                }
                *reinterpret_cast<U*>(un[i].dst + c) = narrow<T, V>(f);
            }
        }
    }
    allow_dependents();
}

template <typename T, int V, bool PAIRED>
cudaError_t launch(const RotaryGeom& g, const void* q, const void* k, const int32_t* pos, const float* inv_freq,
                   void* q_out, void* k_out, cudaStream_t stream) {
    const int units_turn = PAIRED ? g.P / V : (2 * g.P + V - 1) / V;
    const int units_head = PAIRED ? units_turn + (g.d - 2 * g.P) / V : g.d / V;
    const int units_token = (g.heads + g.kv_heads) * units_head;
    // tokens of a CTA: kUnits units a thread, in at least two CTAs for each SM
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const long long spread = (long long)g.B * g.L / (2LL * sms) + 1;
    int per = kUnits * kThreads / units_token;
    if (per > kMaxAngles / g.P) per = kMaxAngles / g.P;
    if (per > kMaxTokens) per = kMaxTokens;
    if (per > g.L) per = g.L;
    if (per > spread) per = (int)spread;
    if (per < 1) per = 1;
    return launch_after_previous(bra_rotary_kernel<T, V, PAIRED>, dim3((unsigned)((g.L + per - 1) / per), (unsigned)g.B),
                                 dim3(kThreads), 0, stream, static_cast<const T*>(q), static_cast<const T*>(k), pos,
                                 inv_freq, static_cast<T*>(q_out), static_cast<T*>(k_out), g, per, units_turn,
                                 divisor(units_token), divisor(units_head), divisor(g.P));
}

}  // namespace

bra_status rotary_launch(const RotaryGeom& g, bool bf16, const void* q, const void* k, const int32_t* pos,
                         const float* inv_freq, void* q_out, void* k_out, cudaStream_t stream) {
    const int v = bf16 ? 8 : 4;
    cudaError_t e;
    // split halves whose P channels are whole vectors move 16 bytes at a time, others one channel
    const bool wide = g.P % v == 0;
    if (g.interleaved)
        e = bf16 ? launch<__nv_bfloat16, 8, false>(g, q, k, pos, inv_freq, q_out, k_out, stream)
                 : launch<float, 4, false>(g, q, k, pos, inv_freq, q_out, k_out, stream);
    else if (wide)
        e = bf16 ? launch<__nv_bfloat16, 8, true>(g, q, k, pos, inv_freq, q_out, k_out, stream)
                 : launch<float, 4, true>(g, q, k, pos, inv_freq, q_out, k_out, stream);
    else
        e = bf16 ? launch<__nv_bfloat16, 1, true>(g, q, k, pos, inv_freq, q_out, k_out, stream)
                 : launch<float, 1, true>(g, q, k, pos, inv_freq, q_out, k_out, stream);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace bra
