// Dropout with the residual's sum, its mask drawn from a counter-based
// generator and never stored:
//   y_i = residual_i + (keep(i / unit) ? x_i / (1 - p) : 0).
// Draw u is word u % 4 of Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011) with the 64-bit key
// ``seed`` and the 64-bit counter ``offset + u / 4``; it keeps its unit where
// the word is at least p 2^32.  The gradient is the same call on dy without
// a residual: the words come again from the same seed and offset, which are
// read from device memory, so that a replayed graph can be given new ones.
//
// Bound by the loads' latency (x and the residual read, y written) and, where every
// element has a draw of its own, by the integer unit as much: the ten rounds cost
// about 15 instructions an element, which keep that unit 52 % busy.  A thread has
// kVectors vectors of eight elements in flight: 12.8 million elements of bf16, 77 MB,
// take 17.5 us (4.4 TB/s) with four, 26 us with one.
#include "kernels.h"
#include "rotary.h"
#include "tma_host.h"

namespace bra {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 4;

__device__ __forceinline__ uint4 philox(uint64_t seed, uint64_t counter) {
    uint32_t x0 = (uint32_t)counter, x1 = (uint32_t)(counter >> 32), x2 = 0u, x3 = 0u;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * x0, b = (uint64_t)0xCD9E8D57u * x2;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
        x1 = (uint32_t)b;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

__device__ __forceinline__ uint32_t word_of(const uint4& w, int i) {
    return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// One element, for the last n % 8.
template <typename T>
__device__ __forceinline__ void one(int64_t i, int64_t unit, uint64_t threshold, float scale, uint64_t seed,
                                    uint64_t offset, const T* x, const T* residual, T* y) {
    const uint64_t u = (uint64_t)(i / unit);
    const bool keep = word_of(philox(seed, offset + u / 4), (int)(u & 3)) >= threshold;
    const float r = residual ? to_f32(residual[i]) : 0.f;
    y[i] = from_f32<T>(keep ? fmaf(to_f32(x[i]), scale, r) : r);
}

// A vector is eight consecutive elements (two counters; or one draw, where a
// unit is a multiple of eight); a CTA's are consecutive, a thread's kThreads apart.
template <typename T, bool SHARED>
__global__ void __launch_bounds__(kThreads)
bra_dropout_add_kernel(const T* x, const T* residual, T* y, int64_t n, int64_t unit, uint64_t threshold, float scale,
                       const uint64_t* rng) {
    constexpr int kWords = sizeof(T) == 2 ? 1 : 2;  // 16-byte words of eight elements
    grid_dependency_wait();
    const int64_t first = ((int64_t)blockIdx.x * kVectors * kThreads + threadIdx.x) * 8;
    uint4 xv[kVectors][kWords], rv[kVectors][kWords];
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
        const int64_t at = first + (int64_t)j * kThreads * 8;
        if (at + 8 > n) continue;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            xv[j][i] = *(reinterpret_cast<const uint4*>(x + at) + i);
            rv[j][i] = residual ? *(reinterpret_cast<const uint4*>(residual + at) + i) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const uint64_t seed = __ldcg(reinterpret_cast<const unsigned long long*>(rng));
    const uint64_t offset = __ldcg(reinterpret_cast<const unsigned long long*>(rng) + 1);
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
        const int64_t at = first + (int64_t)j * kThreads * 8;
        if (at >= n) break;
        if (at + 8 > n) {
            for (int64_t i = at; i < n; ++i) one<T>(i, unit, threshold, scale, seed, offset, x, residual, y);
            break;
        }
        bool keep[8];
        if constexpr (SHARED) {
            const uint64_t u = (uint64_t)(at / unit);
            const bool on = word_of(philox(seed, offset + u / 4), (int)(u & 3)) >= threshold;
#pragma unroll
            for (int i = 0; i < 8; ++i) keep[i] = on;
        } else {
            const uint64_t c = offset + (uint64_t)at / 4;
            const uint4 a = philox(seed, c), b = philox(seed, c + 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                keep[i] = word_of(a, i) >= threshold;
                keep[4 + i] = word_of(b, i) >= threshold;
            }
        }
        float f[8], r[8];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            unpack16(xv[j][i], f + i * (8 / kWords), (const T*)nullptr);
            unpack16(rv[j][i], r + i * (8 / kWords), (const T*)nullptr);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = keep[i] ? fmaf(f[i], scale, r[i]) : r[i];
        if constexpr (sizeof(T) == 2) {
            __nv_bfloat162 h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            *reinterpret_cast<uint4*>(y + at) = *reinterpret_cast<uint4*>(h);
        } else {
            *reinterpret_cast<float4*>(y + at) = make_float4(f[0], f[1], f[2], f[3]);
            *(reinterpret_cast<float4*>(y + at) + 1) = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
    allow_dependents();
}

template <typename T>
cudaError_t launch(int64_t n, int64_t unit, uint64_t threshold, float scale, const uint64_t* rng, const void* x,
                   const void* residual, void* y, cudaStream_t stream) {
    const int64_t grid = ((n + 7) / 8 + kVectors * kThreads - 1) / (kVectors * kThreads);
    auto* kernel = unit == 1 ? bra_dropout_add_kernel<T, false> : bra_dropout_add_kernel<T, true>;
    return launch_after_previous(kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, static_cast<const T*>(x),
                                 static_cast<const T*>(residual), static_cast<T*>(y), n, unit, threshold, scale, rng);
}

}  // namespace

bra_status dropout_add_launch(bool bf16, int64_t n, int64_t unit, uint64_t threshold, float scale,
                              const uint64_t* rng, const void* x, const void* residual, void* y,
                              cudaStream_t stream) {
    const cudaError_t e = bf16 ? launch<__nv_bfloat16>(n, unit, threshold, scale, rng, x, residual, y, stream)
                               : launch<float>(n, unit, threshold, scale, rng, x, residual, y, stream);
    return e == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

}  // namespace bra
