// The gates of the gated linear recurrence and their derivatives.
#pragma once

#include "layer_io.cuh"

namespace kda {
namespace layer {

// Constants of one channel: e = exp(A_log) of its head, bias = dt_bias.
struct GateConst { float e, bias; };

// Decay a = exp(gk) of one token.  Bounded: gk = lb * sigma(e (g + bias)); else
// gk = -e softplus(g + bias), softplus(u) = max(u, 0) + log(1 + exp(-|u|)).
template <bool UB>
__device__ __forceinline__ float gate_decay(float g, GateConst c, float lb) {
    const float u = g + c.bias;
    if (UB) {
        const float sp2 = fmaxf(u, 0.f) * kLog2e + lg2(1.f + ex2(-kLog2e * fabsf(u)));   // softplus * log2(e)
        return ex2(-c.e * sp2);
    }
    return ex2(lb * kLog2e * sigmoid(c.e * u));
}
// The same, with what the derivative needs: slope = d gk / d g, and rate, the factor with
// d gk / d A_log = rate * slope (bounded) or rate (unbounded).
template <bool UB>
__device__ __forceinline__ float gate_slopes(float g, GateConst c, float lb, float &slope, float &dA) {
    const float u = g + c.bias;
    float s, sl;
    if (UB) {
        const float t = ex2(-kLog2e * fabsf(u)), r = rcp(1.f + t);
        // log(1 + t): the series where 1 + t would round the small t away
        const float l1p = t < 0.0078125f ? t * (1.f - t * (0.5f - t * 0.33333333f)) : kLn2 * lg2(1.f + t);
        const float gk = -c.e * (fmaxf(u, 0.f) + l1p);
        s = u >= 0.f ? r : t * r;
        slope = -c.e * s;
        dA = gk;
        return ex2(kLog2e * gk);
    }
    const float z = c.e * u;
    sigmoid_slope(z, s, sl);
    slope = lb * sl * c.e;
    dA = lb * sl * z;
    return ex2(lb * kLog2e * s);
}

}  // namespace layer
}  // namespace kda
