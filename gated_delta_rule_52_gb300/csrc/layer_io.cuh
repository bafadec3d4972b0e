// Typed loads and stores, and the small arithmetic the operators around the delta rule
// share.  All arithmetic on tensor values is fp32; a value is rounded to its tensor's type
// once, when it is stored.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "layer.h"
#include "sm103.cuh"

namespace kda {
namespace layer {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
template <typename E> __device__ __forceinline__ E from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f(float v) { return v; }

// V consecutive elements as one register group; loads and stores of V * sizeof(E) bytes
// (2 to 16, alignment the caller's concern).
template <typename E, int V> struct alignas(sizeof(E) * V) Pack { E e[V]; };

template <typename E, int V>
__device__ __forceinline__ Pack<E, V> ld_pack(const E *p) { return *reinterpret_cast<const Pack<E, V> *>(p); }
// 16-bit values are converted two at a time.
template <typename E, int V>
__device__ __forceinline__ void unpack(const Pack<E, V> &a, float (&f)[V]) {
    if constexpr (sizeof(E) == 2 && V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(a.e)[j / 2];
            if constexpr (std::is_same_v<E, __nv_bfloat16>) {
                f[j] = __uint_as_float(w << 16);
                f[j + 1] = __uint_as_float(w & 0xffff0000u);
            } else {
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                f[j] = t.x, f[j + 1] = t.y;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = to_f(a.e[j]);
    }
}
template <typename E, int V>
__device__ __forceinline__ void ld_f(const E *p, float (&f)[V]) { unpack<E, V>(ld_pack<E, V>(p), f); }
template <typename E, int V>
__device__ __forceinline__ void st_f(E *p, const float (&f)[V]) {
    Pack<E, V> a;
    if constexpr (sizeof(E) == 2 && V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            uint32_t w;
            if constexpr (std::is_same_v<E, __nv_bfloat16>) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f[j + 1]), "f"(f[j]));
            else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f[j + 1]), "f"(f[j]));
            reinterpret_cast<uint32_t *>(a.e)[j / 2] = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) a.e[j] = from_f<E>(f[j]);
    }
    *reinterpret_cast<Pack<E, V> *>(p) = a;
}

// Arithmetic on n values, two per instruction where n is even.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
template <int n>
__device__ __forceinline__ void fma_n(float (&r)[n], const float (&a)[n], const float (&b)[n], const float (&c)[n]) {   // a b + c
    if constexpr (n % 2 == 0) {
#pragma unroll
        for (int j = 0; j < n; j += 2) {
            const float2 t = sm103::fma2(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), make_float2(c[j], c[j + 1]));
            r[j] = t.x, r[j + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j) r[j] = fmaf(a[j], b[j], c[j]);
    }
}
// With the same b and c for all: an immediate operand costs nothing, a register pair of
// constants two moves.
template <int n>
__device__ __forceinline__ void fma_n(float (&r)[n], const float (&a)[n], float b, float c) {
#pragma unroll
    for (int j = 0; j < n; ++j) r[j] = fmaf(a[j], b, c);
}
template <int n>
__device__ __forceinline__ void mul_n(float (&r)[n], const float (&a)[n], const float (&b)[n]) {
    if constexpr (n % 2 == 0) {
#pragma unroll
        for (int j = 0; j < n; j += 2) {
            const float2 t = sm103::mul2(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]));
            r[j] = t.x, r[j + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j) r[j] = a[j] * b[j];
    }
}
template <int n>
__device__ __forceinline__ void add_n(float (&r)[n], const float (&a)[n], const float (&b)[n]) {
    if constexpr (n % 2 == 0) {
#pragma unroll
        for (int j = 0; j < n; j += 2) {
            const float2 t = sm103::add2(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]));
            r[j] = t.x, r[j + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j) r[j] = a[j] + b[j];
    }
}

// Recurrent state of either type.
__device__ __forceinline__ float ld_state(const void *p, int type, int64_t at) {
    return type == kStateBF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at])
                              : static_cast<const float *>(p)[at];
}
__device__ __forceinline__ void st_state(void *p, int type, int64_t at, float v) {
    if (type == kStateBF16) static_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(p)[at] = v;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The smaller of two values, NaN where one is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// sigma(x) = 1 / (1 + e^-x); e^-x overflows to infinity for very negative x, whose
// reciprocal is the right 0.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
// (sigma(-x) with kLog2e as the scale.)
template <int n>
__device__ __forceinline__ void sigmoid_n(float (&s)[n], const float (&x)[n], float scale = -kLog2e) {
    fma_n<n>(s, x, scale, 0.f);
#pragma unroll
    for (int j = 0; j < n; ++j) s[j] = ex2(s[j]);
    fma_n<n>(s, s, 1.f, 1.f);
#pragma unroll
    for (int j = 0; j < n; ++j) s[j] = rcp(s[j]);
}
// First n in [0, N] with cu[n+1] > row (cu non-decreasing, cu[0] = 0): the sequence of a
// packed row.  The result is at most N - 1 whatever cu holds.
__device__ __forceinline__ int64_t seq_of_row(const int64_t *cu, int64_t N, int64_t row) {
    int64_t lo = 0, hi = N - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (cu[mid + 1] > row) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
// Rows [lo, hi) of sequence n, clamped to the packed rows.
template <typename P>
__device__ __forceinline__ void seq_rows(const P &p, int64_t n, int64_t &lo, int64_t &hi) {
    if (p.cu_seqlens) {
        lo = max(p.cu_seqlens[n], (int64_t)0);
        hi = min(p.cu_seqlens[n + 1], p.rows);
    } else {
        lo = n * p.T;
        hi = lo + p.T;
    }
}

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t dtype_bytes(int dtype) { return dtype == kFP32 ? 4 : 2; }

// Calls f with a null pointer of the element type of a dtype code.
template <typename F>
auto with_dtype(int dtype, F &&f) {
    if (dtype == kBF16) return f(static_cast<__nv_bfloat16 *>(nullptr));
    if (dtype == kFP16) return f(static_cast<__half *>(nullptr));
    return f(static_cast<float *>(nullptr));
}

}  // namespace layer
}  // namespace kda
