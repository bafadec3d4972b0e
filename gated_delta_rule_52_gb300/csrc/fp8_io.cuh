// 8-bit floating point: the scale of a block, conversions.
//
// A scale is a power of two, kept as its exponent + 127 in a byte: the smallest one with which
// the block's largest finite magnitude stays within the type's range (448 = 1.75 2^8 in e4m3,
// 57344 = 1.75 2^15 in e5m2).  Multiplying by its inverse is exact, so that the only rounding
// is the one to 8 bits.  Infinities and NaN do not take part in the scale: in e4m3, which has no
// infinity, both become NaN, in e5m2 they stay.
#pragma once

#include "layer_io.cuh"

namespace kda {
namespace layer {

// |x|, or 0 where x is not finite (which is noted).
__device__ __forceinline__ float finite_abs(float x, bool &special) {
    const float a = fabsf(x);
    const bool fine = a < INFINITY;
    special |= !fine;
    return fine ? a : 0.f;
}
// Exponent + 127 of the scale of a block with largest finite magnitude `top`; 127 (a scale of
// 1) where it is below the normal numbers, which count as 0.
__device__ __forceinline__ int scale_byte(float top, bool e5m2) {
    const uint32_t bits = __float_as_uint(top);
    // a mantissa over 1.75 carries into the exponent
    return bits < 0x00800000u ? 127 : max((int)((bits + 0x1fffffu) >> 23) - (e5m2 ? 15 : 8), 1);
}
// 1 / scale, from 2^-120 to 2^126.
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Values times the inverse of a scale.
template <int n>
__device__ __forceinline__ void scale_n(float (&f)[n], float inv) {
    const float2 s = both(inv);
#pragma unroll
    for (int j = 0; j < n; j += 2) {
        const float2 t = sm103::mul2(make_float2(f[j], f[j + 1]), s);
        f[j] = t.x, f[j + 1] = t.y;
    }
}

// Two values to 8 bits each (a in the low byte), rounded to nearest even.
template <bool E5M2>
__device__ __forceinline__ uint32_t pair_to_fp8(float a, float b) {
    uint16_t r;
    if constexpr (E5M2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The conversion saturates; here an infinity becomes what the type has for it.
__device__ __forceinline__ uint32_t with_infinity(uint32_t byte, float v, bool e5m2) {
    if (fabsf(v) != INFINITY) return byte;
    return e5m2 ? 0x7cu | (byte & 0x80u) : 0x7fu;
}
// Four values, `special`: infinities may be among them.
template <bool E5M2>
__device__ __forceinline__ uint32_t quad_to_fp8(float a, float b, float c, float d, bool special) {
    uint32_t r = pair_to_fp8<E5M2>(a, b) | pair_to_fp8<E5M2>(c, d) << 16;
    if (special) {
        const float v[4] = {a, b, c, d};
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) t |= with_infinity(r >> (8 * j) & 0xffu, v[j], E5M2) << (8 * j);
        r = t;
    }
    return r;
}
// The two values of a pair of bytes (exact in 16 bits, hence in 32).
__device__ __forceinline__ float2 pair_from_fp8(uint32_t two, bool e5m2) {
    uint32_t h;
    if (e5m2) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace layer
}  // namespace kda
