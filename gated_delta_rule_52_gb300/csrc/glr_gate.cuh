// The gates of the gated linear recurrence and their derivatives.
#pragma once

#include <cfloat>

#include "layer_io.cuh"
#include "sm103.cuh"

namespace kda {
namespace layer {

// Constants of one channel, folded for base-2 exponentials.  With e = exp(A_log) of its head:
// bounded: k0 = -e log2(e), k1 = k0 dt_bias, so that k0 g + k1 = -log2(e) * e (g + dt_bias);
// else:    k0 = -e,         k1 = log2(e) dt_bias.
struct GateConst { float k0, k1; };


template <bool UB>
__device__ __forceinline__ GateConst gate_const(float A_log, float dt_bias) {
    const float e = expf(A_log);
    return UB ? GateConst{-e, kLog2e * dt_bias} : GateConst{-kLog2e * e, -kLog2e * e * dt_bias};
}

// 2 log2(e) P(z), P the degree-4 Chebyshev fit of atanh(s) / s over z = s^2 in [0, 1/9]
// (relative error 2.2e-8, 6.3e-8 with fp32's own rounding).  With it log2(1 + t) = s * atanh_poly(s^2), s = t / (2 + t), to
// fp32 accuracy relative to the result: lg2(1 + t) would round a small t away, and the sum
// of many small log decays with it.
template <int n>
__device__ __forceinline__ void atanh_poly_n(float (&q)[n], const float (&z)[n]) {
    constexpr float c[4] = {0.40339801f, 0.57743657f, 0.96179163f, 2.88539004f};
    fma_n<n>(q, z, 0.40647438f, c[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) {
        float t[n];
#pragma unroll
        for (int j = 0; j < n; ++j) t[j] = c[k];
        fma_n<n>(q, z, q, t);
    }
}

// 2^x for a log decay x <= 0.  The state keeps a decay's error for 1 / (1 - a) tokens, so near
// 1 it has to be exact to fp32's rounding, which ex2.approx (2^-22) is not: above 2^-0.5 the
// degree-5 polynomial 1 + x P(x), P the Chebyshev fit of (2^x - 1) / x over [-0.5, 0]
// (relative error 1.1e-8, 7.6e-8 with fp32's own rounding).  Errors of the final states of 65536
// tokens against 64 bits: 9.3e-7 without it, 1.7e-7 with it.
template <int n>
__device__ __forceinline__ void exp2_decay_n(float (&a)[n], const float (&x)[n]) {
    constexpr float c[5] = {0.00954248011f, 0.0554907843f, 0.240225688f, 0.693147182f, 1.f};
    float q[n];
    fma_n<n>(q, x, 0.00115564512f, c[0]);
#pragma unroll
    for (int k = 1; k < 5; ++k) {
        float t[n];
#pragma unroll
        for (int j = 0; j < n; ++j) t[j] = c[k];
        fma_n<n>(q, x, q, t);
    }
#pragma unroll
    for (int j = 0; j < n; ++j) a[j] = x[j] > -0.5f ? q[j] : ex2(x[j]);
}

// Decays a = exp(gk) of n tokens or channels.  Bounded: gk = lb sigma(e (g + bias)),
// lb2 = lb log2(e); else gk = -e softplus(g + bias), softplus(u) = max(u, 0) + log(1 + exp(-|u|)).
template <bool UB, int n>
__device__ __forceinline__ void gate_decay_n(float (&a)[n], const float (&g)[n], const float (&k0)[n], const float (&k1)[n], float lb2) {
    float x[n];
    if (UB) {
        float u[n], t[n], s[n], z[n], q[n];
#pragma unroll
        for (int j = 0; j < n; ++j) t[j] = kLog2e;
        fma_n<n>(u, t, g, k1);
#pragma unroll
        for (int j = 0; j < n; ++j) t[j] = ex2(-fabsf(u[j]));
        fma_n<n>(s, t, 1.f, 2.f);
#pragma unroll
        for (int j = 0; j < n; ++j) s[j] = rcp(s[j]), u[j] = fmaxf(u[j], 0.f);
        mul_n<n>(s, t, s);
        mul_n<n>(z, s, s);
        atanh_poly_n<n>(q, z);
        fma_n<n>(x, s, q, u);
        mul_n<n>(x, k0, x);
    } else {
        fma_n<n>(x, k0, g, k1);
#pragma unroll
        for (int j = 0; j < n; ++j) x[j] = ex2(x[j]);
        fma_n<n>(x, x, 1.f, 1.f);
#pragma unroll
        for (int j = 0; j < n; ++j) x[j] = rcp(x[j]);
        fma_n<n>(x, x, lb2, 0.f);
    }
    exp2_decay_n<n>(a, x);
}

// The decays of n tokens or channels again, with what their derivatives are formed from
// later.  Bounded: sigma(z) sigma(-z), with sigma(-z) = e^-z sigma(z), exact relative to itself;
// 1 - sigma(z) would be 1% off at z = 12 and 0 from z = 17 on.  Else sigma(-|g + bias|).
template <bool UB, int n>
__device__ __forceinline__ void decay_and_kept_n(float (&a)[n], float (&kept)[n], const float (&g)[n], const float (&k0)[n],
                                                 const float (&k1)[n], float lb2) {
    float u[n], o[n], x[n];
    if (UB) {
        float t[n], d[n], q[n], z[n];
#pragma unroll
        for (int j = 0; j < n; ++j) z[j] = kLog2e;
        fma_n<n>(u, z, g, k1);
#pragma unroll
        for (int j = 0; j < n; ++j) t[j] = ex2(-fabsf(u[j])), u[j] = fmaxf(u[j], 0.f);
        fma_n<n>(d, t, 1.f, 1.f);
        fma_n<n>(o, t, 1.f, 2.f);
        mul_n<n>(x, d, o);
#pragma unroll
        for (int j = 0; j < n; ++j) x[j] = rcp(x[j]);   // both reciprocals
        mul_n<n>(x, t, x);
        mul_n<n>(kept, x, o);                           // t / (1 + t)
        mul_n<n>(d, x, d);                              // t / (2 + t)
        mul_n<n>(z, d, d);
        atanh_poly_n<n>(q, z);
        fma_n<n>(x, d, q, u);
        mul_n<n>(x, k0, x);
    } else {
        fma_n<n>(u, k0, g, k1);                         // -log2(e) z
        // e^-z held finite: sigma(z) is 0 from 2^126 on, and the product then 0 too, not
        // infinity times 0.  NaN stays.
#pragma unroll
        for (int j = 0; j < n; ++j) u[j] = min_nan(ex2(u[j]), FLT_MAX);
        fma_n<n>(x, u, 1.f, 1.f);
#pragma unroll
        for (int j = 0; j < n; ++j) x[j] = rcp(x[j]);
        mul_n<n>(o, u, x);
        mul_n<n>(kept, x, o);
        fma_n<n>(x, x, lb2, 0.f);
    }
    exp2_decay_n<n>(a, x);
}

// slope = d gk / d g and rate, which times rate_unit is d gk / d A_log, from what was kept.
template <bool UB>
__device__ __forceinline__ float rate_unit(float lb) { return UB ? kLn2 : -kLn2 * lb; }
template <bool UB, int n>
__device__ __forceinline__ void gate_slopes_n(float (&slope)[n], float (&rate)[n], const float (&g)[n], const float (&kept)[n],
                                              const float (&k0)[n], const float (&k1)[n], float lb) {
    float u[n];
    if (UB) {
        // softplus once more: log(1 + t) = -log(1 - m) = 2 atanh(m / (2 - m))
        float o[n], s[n], z[n], q[n];
#pragma unroll
        for (int j = 0; j < n; ++j) z[j] = kLog2e;
        fma_n<n>(u, z, g, k1);
        fma_n<n>(o, kept, -1.f, 1.f);
#pragma unroll
        for (int j = 0; j < n; ++j) o[j] = u[j] >= 0.f ? o[j] : kept[j], u[j] = fmaxf(u[j], 0.f);
        mul_n<n>(slope, k0, o);
        fma_n<n>(s, kept, -1.f, 2.f);
#pragma unroll
        for (int j = 0; j < n; ++j) s[j] = rcp(s[j]);
        mul_n<n>(s, kept, s);
        mul_n<n>(z, s, s);
        atanh_poly_n<n>(q, z);
        fma_n<n>(u, s, q, u);
        mul_n<n>(u, k0, u);
#pragma unroll
        for (int j = 0; j < n; ++j) rate[j] = fmaxf(u[j], -1e30f);   // a decay of 0 times its infinite log is 0
    } else {
        fma_n<n>(u, k0, g, k1);                                      // -log2(e) z
        fma_n<n>(slope, k0, rate_unit<UB>(lb), 0.f);
        mul_n<n>(slope, slope, kept);
        mul_n<n>(rate, kept, u);
#pragma unroll
        for (int j = 0; j < n; ++j) rate[j] = kept[j] == 0.f ? 0.f : rate[j];   // so is a slope of 0 times an infinite argument
    }
}

}  // namespace layer
}  // namespace kda
