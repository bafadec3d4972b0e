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
// (relative error 8e-9).
__device__ __forceinline__ float atanh_poly(float z) {
    return fmaf(z, fmaf(z, fmaf(z, fmaf(z, 0.40647438f, 0.40339801f), 0.57743657f), 0.96179163f), 2.88539004f);
}
// log2(1 + t) for t in [0, 1], to fp32 accuracy relative to the result (lg2(1 + t) rounds
// a small t away, and the sum of many small log decays with it): with s = t / (2 + t),
// log(1 + t) = 2 atanh(s).
__device__ __forceinline__ float log2_1p(float t) {
    const float s = t * rcp(2.f + t), z = s * s;
    return s * atanh_poly(z);
}

// 2^x for a log decay x <= 0.  The state keeps a decay's error for 1 / (1 - a) tokens, so near
// 1 it has to be exact to fp32's rounding, which ex2.approx (2^-22) is not: above 2^-0.5 the
// degree-5 polynomial 1 + x P(x), P the Chebyshev fit of (2^x - 1) / x over [-0.5, 0]
// (relative error 7e-8 with fp32's own rounding).  Errors of the final states of 65536
// tokens against 64 bits: 9.3e-7 without it, 1.7e-7 with it.
__device__ __forceinline__ float2 exp2_decay2(float2 x) {
    using namespace sm103;
    const auto c = [](float v) { return make_float2(v, v); };
    float2 q = fma2(x, c(0.00115564512f), c(0.00954248011f));
    q = fma2(x, q, c(0.0554907843f));
    q = fma2(x, q, c(0.240225688f));
    q = fma2(x, q, c(0.693147182f));
    q = fma2(x, q, c(1.f));
    return make_float2(x.x > -0.5f ? q.x : ex2(x.x), x.y > -0.5f ? q.y : ex2(x.y));
}
__device__ __forceinline__ float exp2_decay(float x) {
    const float q = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, 0.00115564512f, 0.00954248011f), 0.0554907843f), 0.240225688f),
                                 0.693147182f), 1.f);
    return x > -0.5f ? q : ex2(x);
}

// Decay a = exp(gk) of one token.  Bounded: gk = lb sigma(e (g + bias)), lb2 = lb log2(e);
// else gk = -e softplus(g + bias), softplus(u) = max(u, 0) + log(1 + exp(-|u|)).
template <bool UB>
__device__ __forceinline__ float gate_decay(float g, GateConst c, float lb2) {
    if (UB) {
        const float u2 = fmaf(kLog2e, g, c.k1);
        return exp2_decay(c.k0 * (fmaxf(u2, 0.f) + log2_1p(ex2(-fabsf(u2)))));
    }
    return exp2_decay(lb2 * rcp(1.f + ex2(fmaf(c.k0, g, c.k1))));
}
// Two tokens or channels at a time (packed fp32 arithmetic).
template <bool UB>
__device__ __forceinline__ float2 gate_decay2(float2 g, GateConst c0, GateConst c1, float lb2) {
    using namespace sm103;
    const float2 k0 = make_float2(c0.k0, c1.k0), k1 = make_float2(c0.k1, c1.k1), one = make_float2(1.f, 1.f);
    if (UB) {
        const float2 u2 = fma2(make_float2(kLog2e, kLog2e), g, k1);
        const float2 t = make_float2(ex2(-fabsf(u2.x)), ex2(-fabsf(u2.y)));
        const float2 d = add2(t, make_float2(2.f, 2.f));
        const float2 s = mul2(t, make_float2(rcp(d.x), rcp(d.y))), z = mul2(s, s);
        float2 q = fma2(z, make_float2(0.40647438f, 0.40647438f), make_float2(0.40339801f, 0.40339801f));
        q = fma2(z, q, make_float2(0.57743657f, 0.57743657f));
        q = fma2(z, q, make_float2(0.96179163f, 0.96179163f));
        q = fma2(z, q, make_float2(2.88539004f, 2.88539004f));
        const float2 gk = mul2(k0, fma2(s, q, make_float2(fmaxf(u2.x, 0.f), fmaxf(u2.y, 0.f))));
        return exp2_decay2(gk);
    }
    const float2 z2 = fma2(k0, g, k1);
    const float2 d = add2(make_float2(ex2(z2.x), ex2(z2.y)), one);
    const float2 gk = mul2(make_float2(lb2, lb2), make_float2(rcp(d.x), rcp(d.y)));
    return exp2_decay2(gk);
}
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    using namespace sm103;
    const float2 m = mul2(make_float2(-kLog2e, -kLog2e), x);
    const float2 d = add2(make_float2(ex2(m.x), ex2(m.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}
// What the derivatives of one token are formed from, kept between the two halves of the
// backward pass: `gate` is the decay a (bounded) or its log2 (else), `mg` and `mi` the
// smaller of sigma(v) and sigma(-v) for the gate's argument and for i.  The smaller one is
// exact relative to itself, and with it both sigma and its slope m (1 - m).
struct TokenGates { float gate, mg, mi; };

template <bool UB>
__device__ __forceinline__ TokenGates token_gates(float g, float i, GateConst c, float lb2, float &a, float &s) {
    const float ti = ex2(-kLog2e * fabsf(i)), mi = ti * rcp(1.f + ti);
    s = i >= 0.f ? 1.f - mi : mi;
    if (UB) {
        const float u2 = fmaf(kLog2e, g, c.k1);
        const float t = ex2(-fabsf(u2)), d1 = 1.f + t, d2 = 2.f + t, r = rcp(d1 * d2);   // both reciprocals
        const float q = t * d1 * r;                                                     // t / (2 + t)
        const float gk2 = c.k0 * fmaf(q, atanh_poly(q * q), fmaxf(u2, 0.f));
        a = exp2_decay(gk2);
        return {gk2, t * d2 * r, mi};
    }
    const float z2 = fmaf(c.k0, g, c.k1);   // -log2(e) z
    const float t = ex2(-fabsf(z2)), mg = t * rcp(1.f + t);
    a = exp2_decay(lb2 * (z2 <= 0.f ? 1.f - mg : mg));
    return {a, mg, mi};
}
// slope = d gk / d g, rate = d gk / d A_log, from the same token's kept values.
template <bool UB>
__device__ __forceinline__ void gate_slopes(float g, GateConst c, float lb, const TokenGates &k, float &slope, float &rate) {
    if (UB) {
        const float u2 = fmaf(kLog2e, g, c.k1);
        slope = c.k0 * (u2 >= 0.f ? 1.f - k.mg : k.mg);
        rate = kLn2 * fmaxf(k.gate, -1e30f);   // a decay of 0 times its infinite log is 0
    } else {
        const float z2 = fmaf(c.k0, g, c.k1), l = -kLn2 * lb * (k.mg - k.mg * k.mg);   // -ln 2 lb sigma'
        slope = l * c.k0;
        rate = l == 0.f ? 0.f : l * z2;       // so is a slope of 0 times an infinite argument
    }
}

}  // namespace layer
}  // namespace kda
