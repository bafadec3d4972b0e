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

// log2(1 + t) for t in [0, 1], to fp32 accuracy relative to the result (lg2(1 + t) rounds
// a small t away, and the sum of many small log decays with it): with s = t / (2 + t),
// log(1 + t) = 2 atanh(s) = 2 s P(s^2), P the degree-4 Chebyshev fit of atanh(s) / s over
// s^2 in [0, 1/9] (relative error 8e-9).
__device__ __forceinline__ float log2_1p(float t) {
    const float s = t * rcp(2.f + t), z = s * s;
    const float q = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 0.40647438f, 0.40339801f), 0.57743657f), 0.96179163f), 2.88539004f);
    return s * q;
}

// Decay a = exp(gk) of one token.  Bounded: gk = lb sigma(e (g + bias)), lb2 = lb log2(e);
// else gk = -e softplus(g + bias), softplus(u) = max(u, 0) + log(1 + exp(-|u|)).
template <bool UB>
__device__ __forceinline__ float gate_decay(float g, GateConst c, float lb2) {
    if (UB) {
        const float u2 = fmaf(kLog2e, g, c.k1);
        return ex2(c.k0 * (fmaxf(u2, 0.f) + log2_1p(ex2(-fabsf(u2)))));
    }
    return ex2(lb2 * rcp(1.f + ex2(fmaf(c.k0, g, c.k1))));
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
        return make_float2(ex2(gk.x), ex2(gk.y));
    }
    const float2 z2 = fma2(k0, g, k1);
    const float2 d = add2(make_float2(ex2(z2.x), ex2(z2.y)), one);
    const float2 gk = mul2(make_float2(lb2, lb2), make_float2(rcp(d.x), rcp(d.y)));
    return make_float2(ex2(gk.x), ex2(gk.y));
}
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    using namespace sm103;
    const float2 m = mul2(make_float2(-kLog2e, -kLog2e), x);
    const float2 d = add2(make_float2(ex2(m.x), ex2(m.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}
// The same, with what the derivative needs: slope = d gk / d g, and rate, d gk / d A_log.
template <bool UB>
__device__ __forceinline__ float gate_slopes(float g, GateConst c, float lb2, float &slope, float &rate) {
    if (UB) {
        const float u2 = fmaf(kLog2e, g, c.k1);
        const float t = ex2(-fabsf(u2)), r = rcp(1.f + t);
        const float gk2 = c.k0 * (fmaxf(u2, 0.f) + log2_1p(t));
        slope = c.k0 * (u2 >= 0.f ? r : t * r);
        rate = kLn2 * gk2;
        return ex2(gk2);
    }
    const float z2 = fmaf(c.k0, g, c.k1);   // -log2(e) z
    const float t = ex2(-fabsf(z2)), r = rcp(1.f + t), tr = t * r;
    const float lsl = lb2 * tr * r;         // lb2 sigma'(z)
    slope = -lsl * c.k0 * (kLn2 * kLn2);    // lb sigma'(z) e
    rate = -lsl * z2 * (kLn2 * kLn2);       // lb sigma'(z) z
    return ex2(lb2 * (z2 <= 0.f ? r : tr));
}

}  // namespace layer
}  // namespace kda
