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
// Bound by HBM: Q and K are read and written once, in 16-byte vectors; a
// thread's loads are issued before the CTA's angles are formed.
#include "kernels.h"
#include "rotary.h"
#include "tma_host.h"

namespace bra {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 2048;  // (token, pair) angles of a CTA: 16 KB of shared memory

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
bra_rotary_kernel(const T* __restrict__ q, const T* __restrict__ k, const int32_t* __restrict__ pos,
                  const float* __restrict__ inv_freq, T* __restrict__ qo, T* __restrict__ ko, RotaryGeom g,
                  int tokens_per_cta, int units_turn, int units_head) {
    using U = typename Vec<T, V>::type;
    __shared__ float2 table[kMaxAngles];
    const long long tokens = (long long)g.B * g.L;
    const long long token0 = (long long)blockIdx.x * tokens_per_cta;
    const int here = (int)min((long long)tokens_per_cta, tokens - token0);
    grid_dependency_wait();

    for (int e = threadIdx.x; e < here * g.P; e += kThreads) {
        const int tk = e / g.P, i = e - tk * g.P;
        const long long at = token0 + tk;
        const int b = (int)(at / g.L), l = (int)(at - (long long)b * g.L);
        const int axis = i < g.axis1 ? 0 : (i < g.axis2 ? 1 : 2);
        int p;
        if (pos) {
            p = __ldcg(pos + (size_t)b * g.pos_batch + (size_t)l * 3 + axis);
        } else {
            const int row = l / g.W;
            p = axis == 2 ? l - row * g.W : (axis == 1 ? row % g.H : row / g.H);
        }
        // turns, reduced to [-1/2, 1/2]
        double turns = (double)p * (double)__ldcg(inv_freq + i) * 0.15915494309189533577;
        turns -= rint(turns);
        float s, c;
        sincospif(2.f * (float)turns, &s, &c);
        table[e] = make_float2(c, g.inverse ? -s : s);
    }
    __syncthreads();

    const int heads = g.heads + g.kv_heads, per_token = heads * units_head;
    for (int u = threadIdx.x; u < here * per_token; u += kThreads) {
        const int tk = u / per_token, w = u - tk * per_token, head = w / units_head, x = w - head * units_head;
        const long long at = token0 + tk;
        const int b = (int)(at / g.L), l = (int)(at - (long long)b * g.L);
        const T* src;
        T* dst;
        if (head < g.heads) {
            src = q + (size_t)b * g.q_batch + (size_t)l * g.q_row + (size_t)head * g.d;
            dst = qo + (size_t)b * g.qo_batch + (size_t)l * g.qo_row + (size_t)head * g.d;
        } else {
            src = k + (size_t)b * g.k_batch + (size_t)l * g.k_row + (size_t)(head - g.heads) * g.d;
            dst = ko + (size_t)b * g.ko_batch + (size_t)l * g.ko_row + (size_t)(head - g.heads) * g.d;
        }
        const float2* tab = table + tk * g.P;
        if constexpr (PAIRED) {
            if (x < units_turn) {
                const int c = x * V;
                const U a = *reinterpret_cast<const U*>(src + c), z = *reinterpret_cast<const U*>(src + g.P + c);
                float f[V], h[V];
                widen<T, V>(a, f);
                widen<T, V>(z, h);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 t = tab[c + i];
                    const float y = f[i] * t.x - h[i] * t.y;
                    h[i] = h[i] * t.x + f[i] * t.y;
                    f[i] = y;
                }
                *reinterpret_cast<U*>(dst + c) = narrow<T, V>(f);
                *reinterpret_cast<U*>(dst + g.P + c) = narrow<T, V>(h);
            } else {
                const int c = 2 * g.P + (x - units_turn) * V;
                *reinterpret_cast<U*>(dst + c) = *reinterpret_cast<const U*>(src + c);
            }
        } else {
            const int c = x * V;
            U a = *reinterpret_cast<const U*>(src + c);
            if (x < units_turn) {
                float f[V];
                widen<T, V>(a, f);
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    if ((c + i) / 2 >= g.P) continue;
                    const float2 t = tab[(c + i) / 2];
                    const float y = f[i] * t.x - f[i + 1] * t.y;
                    f[i + 1] = f[i + 1] * t.x + f[i] * t.y;
                    f[i] = y;
                }
                a = narrow<T, V>(f);
            }
            *reinterpret_cast<U*>(dst + c) = a;
        }
    }
    allow_dependents();
}

template <typename T, int V, bool PAIRED>
cudaError_t launch(const RotaryGeom& g, const void* q, const void* k, const int32_t* pos, const float* inv_freq,
                   void* q_out, void* k_out, cudaStream_t stream) {
    const int units_turn = PAIRED ? g.P / V : (2 * g.P + V - 1) / V;
    const int units_head = PAIRED ? units_turn + (g.d - 2 * g.P) / V : g.d / V;
    int per = kMaxAngles / g.P;
    const int want = (2 * kThreads) / ((g.heads + g.kv_heads) * units_head);  // two units a thread
    if (per > want) per = want > 0 ? want : 1;
    const long long tokens = (long long)g.B * g.L;
    const long long grid = (tokens + per - 1) / per;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_after_previous(bra_rotary_kernel<T, V, PAIRED>, dim3((unsigned)grid), dim3(kThreads), 0, stream,
                                 static_cast<const T*>(q), static_cast<const T*>(k), pos, inv_freq,
                                 static_cast<T*>(q_out), static_cast<T*>(k_out), g, per, units_turn, units_head);
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
