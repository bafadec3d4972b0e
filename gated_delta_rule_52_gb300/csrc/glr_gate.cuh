// The gates of the gated linear recurrence and their derivatives.
#pragma once

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
// (relative error 8e-9).  With it log2(1 + t) = s * atanh_poly(s^2), s = t / (2 + t), to
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
// (relative error 7e-8 with fp32's own rounding).  Errors of the final states of 65536
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

// The same and sigma(i) of n tokens or channels, with two values each that their derivatives
// are formed from later, kept_g and kept_i.  EXACT (tensors in 32 bits): the smaller of
// sigma(v) and sigma(-v), which is exact relative to itself, and with it sigma and its slope
// m (1 - m) at any v.  Else (tensors in 16 bits): sigma(v) itself; 1 - sigma is then off by
// 2^-24, below the rounding of a 16-bit gradient while 1 - sigma is above 2^-13.  (The gate
// without a lower bound keeps the smaller one in either case: its softplus needs it.)
template <bool UB, bool EXACT, int n>
__device__ __forceinline__ void token_gates_n(float (&a)[n], float (&s)[n], float (&kept_g)[n], float (&kept_i)[n],
                                              const float (&g)[n], const float (&i)[n], const float (&k0)[n],
                                              const float (&k1)[n], float lb2) {
    float t[n], d[n], o[n], u[n], x[n];
    if (EXACT) {
#pragma unroll
        for (int j = 0; j < n; ++j) t[j] = ex2(-kLog2e * fabsf(i[j]));
        fma_n<n>(d, t, 1.f, 1.f);
#pragma unroll
        for (int j = 0; j < n; ++j) d[j] = rcp(d[j]);
        mul_n<n>(kept_i, t, d);
        fma_n<n>(o, kept_i, -1.f, 1.f);
#pragma unroll
        for (int j = 0; j < n; ++j) s[j] = i[j] >= 0.f ? o[j] : kept_i[j];
    } else {
        sigmoid_n<n>(s, i);
#pragma unroll
        for (int j = 0; j < n; ++j) kept_i[j] = s[j];
    }
    if (UB) {
        float q[n], z[n];
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
        mul_n<n>(kept_g, x, o);                         // t / (1 + t)
        mul_n<n>(d, x, d);                              // t / (2 + t)
        mul_n<n>(z, d, d);
        atanh_poly_n<n>(q, z);
        fma_n<n>(x, d, q, u);
        mul_n<n>(x, k0, x);
    } else {
        fma_n<n>(u, k0, g, k1);                         // -log2(e) z
        if (EXACT) {
#pragma unroll
            for (int j = 0; j < n; ++j) t[j] = ex2(-fabsf(u[j]));
            fma_n<n>(d, t, 1.f, 1.f);
#pragma unroll
            for (int j = 0; j < n; ++j) d[j] = rcp(d[j]);
            mul_n<n>(kept_g, t, d);
            fma_n<n>(o, kept_g, -1.f, 1.f);
#pragma unroll
            for (int j = 0; j < n; ++j) x[j] = u[j] <= 0.f ? o[j] : kept_g[j];
        } else {
#pragma unroll
            for (int j = 0; j < n; ++j) t[j] = ex2(u[j]);
            fma_n<n>(d, t, 1.f, 1.f);
#pragma unroll
            for (int j = 0; j < n; ++j) x[j] = kept_g[j] = rcp(d[j]);
        }
        fma_n<n>(x, x, lb2, 0.f);
    }
    exp2_decay_n<n>(a, x);
}

// sigma(i), sigma(-i) from kept_i.
template <bool EXACT, int n>
__device__ __forceinline__ void input_gates_n(float (&s)[n], float (&o)[n], const float (&i)[n], const float (&kept)[n]) {
    fma_n<n>(o, kept, -1.f, 1.f);
#pragma unroll
    for (int j = 0; j < n; ++j) {
        const float m = kept[j], r = o[j];
        s[j] = !EXACT || i[j] < 0.f ? m : r;
        o[j] = !EXACT || i[j] < 0.f ? r : m;
    }
}
// slope = d gk / d g and rate = d gk / d A_log from kept_g.
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
        for (int j = 0; j < n; ++j) rate[j] = kLn2 * fmaxf(u[j], -1e30f);   // a decay of 0 times its infinite log is 0
    } else {
        float l[n], o[n];
        fma_n<n>(u, k0, g, k1);
        fma_n<n>(o, kept, -1.f, 1.f);
        mul_n<n>(l, kept, o);
        fma_n<n>(l, l, -kLn2 * lb, 0.f);                                    // -ln 2 lb sigma'
        mul_n<n>(slope, l, k0);
        mul_n<n>(rate, l, u);
#pragma unroll
        for (int j = 0; j < n; ++j) rate[j] = l[j] == 0.f ? 0.f : rate[j];  // so is a slope of 0 times an infinite argument
    }
}

}  // namespace layer
}  // namespace kda
