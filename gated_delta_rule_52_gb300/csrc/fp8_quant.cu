// Quantisation to 8 bits with a power-of-two scale for each block of 128 (fp8_io.cuh), and back.
//   q = x / s,  s = 2^e for 128 neighbours of a row, or for a tile of 128 rows by 128 columns
// The transposed result has its blocks along the columns.  A CTA takes a tile of 128 x 128,
// which holds every block that it touches: the tile is read once, into registers, and both
// results come from there, the transposed one by way of shared memory.
//
// 8192 x 8192 bf16: one way 36.7 us (81% of the copy rate), both ways 50.8 us (78%), by tiles 45.4 us
// (88%); 8192 x 2048 fp32 by tiles both ways 20 us (75%), 8192 x 8192 67 us (89%).  Bound by issue (74% of
// the slots: a row's and a column's maximum, two scalings and two conversions per element); in 32 bits
// by memory, and of few tiles by rounds: 1024 CTAs on 304 places are 3.4, which take 4, and a CTA loads
// no further tile while it stores.  Unaligned rows are loaded and stored element by element (8192 x 8191 both ways 92 us).
// Back: 8192 x 8192 to bf16 31.2 us (96%).
#include <algorithm>

#include "fp8_io.cuh"
#include "layer_copy.cuh"

namespace kda {
namespace {

using namespace layer;

constexpr int kTile = kFp8Block;
// Threads of a CTA, and groups of 64 rows that a thread has rows of: 16-bit tiles with 64 elements per
// thread and 4 CTAs per SM (8192 x 8192 bf16 both ways 50 us; 65 us with 32 elements), 32-bit ones with
// 32 and 2 (8192 x 2048 20 us; 22 us with 64).
template <typename E> constexpr int kQuantThreads = sizeof(E) == 2 ? 256 : 512;
template <typename E> constexpr int kHalves = 512 / kQuantThreads<E>;

// 8 neighbours as they are in memory, two 16-bit elements to a word.  Their magnitudes compare like
// the integers that their bits are; with kShift added infinity and NaN leave the positive signed
// numbers, so that a signed maximum passes over them.
template <typename E>
struct Eight {
    static constexpr int kWords = sizeof(E) * 2;
    static constexpr bool kPairs = sizeof(E) == 2;
    static constexpr uint32_t kMask = kPairs ? 0x7fff7fffu : 0x7fffffffu;
    static constexpr uint32_t kShift = std::is_same_v<E, __half> ? 0x04000400u : kPairs ? 0x00800080u : 0x00800000u;   // 0
    static constexpr uint32_t kSigns = kPairs ? 0x80008000u : 0x80000000u;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const E *p) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 t = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(p) + i);
            w[i] = t.x, w[i + 1] = t.y, w[i + 2] = t.z, w[i + 3] = t.w;
        }
    }
    __device__ __forceinline__ void load(const E *p, int n) {   // the first n, zeros behind them
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) continue;
            if constexpr (kPairs) w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[j] << (16 * (j & 1));
            else w[j] = reinterpret_cast<const uint32_t *>(p)[j];
        }
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        if constexpr (kPairs) {
            unpack<E, 8>(*reinterpret_cast<const Pack<E, 8> *>(w), f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
        }
    }
    __device__ __forceinline__ float2 two(int j) const {   // elements j and j + 1, j even
        if constexpr (std::is_same_v<E, __nv_bfloat16>) return sm103::bf16x2_to_f2(w[j / 2]);
        else if constexpr (kPairs) return __half22float2(reinterpret_cast<const __half2 *>(w)[j / 2]);
        else return make_float2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
    }
    __device__ __forceinline__ uint32_t magnitude(int i) const { return (w[i] & kMask) + kShift; }
};
template <typename E>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (sizeof(E) == 2) asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else r = (uint32_t)max((int)a, (int)b);
    return r;
}
// The number that a shifted magnitude (of 16 bits: the low half of a word) is.
template <typename E>
__device__ __forceinline__ float number(uint32_t m) {
    if constexpr (sizeof(E) == 2) return to_f(__builtin_bit_cast(E, (uint16_t)(m - (Eight<E>::kShift & 0xffffu))));
    else return __uint_as_float(m - Eight<E>::kShift);
}

// Thread t: columns 8 (t % 16) .. + 7 of rows 64 h + 4 (t / 16) + i, kept as they are loaded.
template <typename E, bool E5M2, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads<E>, sizeof(E) == 2 ? 4 : 2) quantize_kernel(QuantParams p) {
    using Group = Eight<E>;
    constexpr int kWords = Group::kWords, kWarps = kQuantThreads<E> / 32, kH = kHalves<E>;
    __shared__ uint32_t tops[kWarps][kWords * 16];
    __shared__ uint32_t warp_top[4];
    __shared__ uint8_t col_scale[kTile];
    __shared__ uint32_t turned[kTile * kTile / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const uint32_t across = (uint32_t)ceil_div(p.cols, kTile), br = blockIdx.x / across, bc = blockIdx.x - br * across;
    const int64_t r0 = (int64_t)br * kTile, c0 = (int64_t)bc * kTile, c = c0 + 8 * cg;
    const int cols = (int)min(max(p.cols - c, (int64_t)0), (int64_t)8), rows = (int)min(p.rows - r0, (int64_t)kTile);
    Group v[kH][4];
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    {
        const E *at = static_cast<const E *>(p.x) + (r0 + 4 * rg) * p.xs + c;
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 64 * h + 4 * rg + i, n = r < rows ? cols : 0;
                if (WIDE && n == 8) v[h][i].load(at + (64 * h + i) * p.xs);
                else v[h][i].load(at + (64 * h + i) * p.xs, n);
            }
    }
    uint32_t row_top[kH][4], col_top[kWords], any = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) col_top[w] = Group::kShift;
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t = Group::kShift;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                const uint32_t m = v[h][i].magnitude(w);
                any |= m;
                t = larger<E>(t, m);
                col_top[w] = larger<E>(col_top[w], m);
            }
            row_top[h][i] = Group::kPairs ? larger<E>(t, t >> 16) : t;
        }
    const bool special = __any_sync(0xffffffffu, (any & Group::kSigns) != 0);   // the warp holds infinities or NaN
    if (p.qt || p.tile) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const uint32_t t = larger<E>(col_top[w], __shfl_xor_sync(0xffffffffu, col_top[w], 16));
            if (lane < 16) tops[warp][cg * kWords + w] = t;
        }
        __syncthreads();
        if (threadIdx.x < kTile) {
            // column threadIdx.x: half a word of a 16-bit type
            const int word = Group::kPairs ? threadIdx.x >> 1 : threadIdx.x;
            uint32_t t = tops[0][word];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) t = larger<E>(t, tops[w][word]);
            if (Group::kPairs) t = threadIdx.x & 1 ? t >> 16 : t & 0xffffu;
            if (p.tile) {
                t = __reduce_max_sync(0xffffffffu, t);   // positive: kShift or more
                if (lane == 0) warp_top[warp] = t;
            } else {
                col_scale[threadIdx.x] = (uint8_t)scale_byte(number<E>(t), E5M2);
            }
        }
        __syncthreads();
    }
    int tile_scale = 0;
    if (p.tile) {
        tile_scale = scale_byte(number<E>(max(max(warp_top[0], warp_top[1]), max(warp_top[2], warp_top[3]))), E5M2);
        if (threadIdx.x == 0) {
            if (p.q) p.s[br * p.ss + bc] = (uint8_t)tile_scale;
            if (p.qt) p.st[bc * p.sts + br] = (uint8_t)tile_scale;
        }
    }
    // maxima of the rows over the 16 lanes that share them, 16-bit ones two rows to a word
    if (p.q && !p.tile) {
#pragma unroll
        for (int h = 0; h < kH; ++h) {
            constexpr int n = Group::kPairs ? 2 : 4;
            uint32_t t[n];
#pragma unroll
            for (int i = 0; i < n; ++i) t[i] = Group::kPairs ? (row_top[h][2 * i] & 0xffffu) | row_top[h][(2 * i + 1) & 3] << 16 : row_top[h][i];
#pragma unroll
            for (int o = 8; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) t[i] = larger<E>(t[i], __shfl_xor_sync(0xffffffffu, t[i], o));
#pragma unroll
            for (int i = 0; i < 4; ++i) row_top[h][i] = Group::kPairs ? (i & 1 ? t[i / 2] >> 16 : t[i / 2] & 0xffffu) : t[i % n];
        }
    }
    // to 8 bits, with a path of its own for infinities and NaN
    const auto convert = [&](auto with_special) {
        constexpr bool kSpecial = decltype(with_special)::value;
        if (p.q) {
            const bool whole = cols == 8 && p.qs % 8 == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0;
            uint8_t *first = static_cast<uint8_t *>(p.q) + (r0 + 4 * rg) * p.qs + c;
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = p.tile ? tile_scale : scale_byte(number<E>(row_top[h][i]), E5M2);
                    const int r = 64 * h + 4 * rg + i;
                    if (r >= rows || cols == 0) continue;
                    if (!p.tile && cg == 0) p.s[(r0 + r) * p.ss + bc] = (uint8_t)e;
                    float f[8];
                    v[h][i].values(f);
                    scale_n(f, inverse_scale(e));
                    const uint32_t lo = quad_to_fp8<E5M2>(f[0], f[1], f[2], f[3], kSpecial), hi = quad_to_fp8<E5M2>(f[4], f[5], f[6], f[7], kSpecial);
                    uint8_t *at = first + (64 * h + i) * p.qs;
                    if (whole) {
                        *reinterpret_cast<uint2 *>(at) = make_uint2(lo, hi);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < cols) at[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
                    }
                }
        }
        if (!p.qt) return;
        // four rows of a column are one word; word w of column c stands at place w + 2 (c / 8) of
        // its line, so that a warp's words lie in 32 banks
#pragma unroll
        for (int j = 0; j < 8; j += 2) {                      // two columns at a time
            float2 inv;
            inv.x = inverse_scale(p.tile ? tile_scale : col_scale[8 * cg + j]);
            inv.y = inverse_scale(p.tile ? tile_scale : col_scale[8 * cg + j + 1]);
#pragma unroll
            for (int h = 0; h < kH; ++h) {
                float2 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = sm103::mul2(v[h][i].two(j), inv);
                uint32_t *to = &turned[(8 * cg + j) * 32 + ((16 * h + rg + 2 * cg) & 31)];
                to[0] = quad_to_fp8<E5M2>(f[0].x, f[1].x, f[2].x, f[3].x, kSpecial);
                to[32] = quad_to_fp8<E5M2>(f[0].y, f[1].y, f[2].y, f[3].y, kSpecial);
            }
        }
    };
    if (special) convert(std::true_type{});
    else convert(std::false_type{});
    if (!p.qt) return;
    __syncthreads();
    // 8 lanes to a column, 16 rows each
    const bool words = p.qts % 16 == 0 && reinterpret_cast<uintptr_t>(p.qt) % 16 == 0;
    const int w0 = 4 * (lane & 7), n = min(rows - 4 * w0, 16);
#pragma unroll
    for (int k = 0; k < kTile / 4 / kWarps; ++k) {
        const int col = 4 * (kWarps * k + warp) + (lane >> 3);
        if (c0 + col >= p.cols) continue;
        const int turn = 2 * (col >> 3);
        const uint2 a = *reinterpret_cast<const uint2 *>(&turned[col * 32 + ((w0 + turn) & 31)]);
        const uint2 b = *reinterpret_cast<const uint2 *>(&turned[col * 32 + ((w0 + 2 + turn) & 31)]);
        uint8_t *at = static_cast<uint8_t *>(p.qt) + (c0 + col) * p.qts + r0 + 4 * w0;
        if (words && n == 16) {
            *reinterpret_cast<uint4 *>(at) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            const uint32_t t[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < n) at[j] = (uint8_t)(t[j / 4] >> (8 * (j & 3)));
        }
        if (!p.tile && (lane & 7) == 0) p.st[(c0 + col) * p.sts + br] = col_scale[col];
    }
}

// Scale of a byte: 2^(byte - 127), NaN for 255.  (2^-127, which is below the normal numbers,
// only where a caller wrote a 0.)
__device__ __forceinline__ float scale_of(int byte) {
    return byte == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)max(byte, 1) << 23);
}

// A warp takes kTurns pieces of 32 V neighbouring elements of a row, V to a lane.
constexpr int kTurns = 4;

template <typename E, int V>
__global__ void __launch_bounds__(256) dequantize_kernel(QuantParams p, uint32_t pieces) {
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    const bool e5m2 = p.q_dtype == kE5M2;
    const uint32_t item = blockIdx.x * 8 + (threadIdx.x >> 5), row = item / pieces;
    if (row >= p.rows) return;
    const int64_t r = row, first = (int64_t)(item - row * pieces) * (32 * V * kTurns) + (threadIdx.x & 31) * V;
    const uint8_t *q = static_cast<const uint8_t *>(p.q) + r * p.qs, *s = p.s + (p.tile ? r / kTile : r) * p.ss;
    E *out = static_cast<E *>(const_cast<void *>(p.x)) + r * p.xs;
    Pack<uint8_t, V> in[kTurns];
    uint8_t scale[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int64_t c = first + k * 32 * V;
        if (c < p.cols) in[k] = *reinterpret_cast<const Pack<uint8_t, V> *>(q + c), scale[k] = s[c / kTile];
    }
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int64_t c = first + k * 32 * V;
        if (c >= p.cols) break;
        const int byte = scale[k];
        const float f = scale_of(byte), half = byte == 0 ? 0.5f : 1.f;
        if constexpr (V == 1) {
            out[c] = from_f<E>(pair_from_fp8(in[k].e[0], e5m2).x * half * f);
        } else {
            float v[V];
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float2 t = pair_from_fp8(reinterpret_cast<const uint16_t *>(in[k].e)[j / 2], e5m2);
                v[j] = t.x * half * f, v[j + 1] = t.y * half * f;
            }
            constexpr int P = 16 / sizeof(E);
#pragma unroll
            for (int j = 0; j < V; j += P) st_f<E, P>(out + c + j, reinterpret_cast<const float (&)[P]>(v[j]));
        }
    }
}

}  // namespace

cudaError_t launch_quantize(const QuantParams &p, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const int64_t grid = ceil_div(p.cols, kTile) * ceil_div(p.rows, kTile);
        const bool wide = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.xs % (16 / sizeof(E)) == 0;
        const auto run = [&](auto kernel) { return launch_early(kernel, grid, dim3(kQuantThreads<E>), 0, stream, 0, p); };
        if (p.q_dtype == kE5M2) return wide ? run(quantize_kernel<E, true, true>) : run(quantize_kernel<E, true, false>);
        return wide ? run(quantize_kernel<E, false, true>) : run(quantize_kernel<E, false, false>);
    });
}

cudaError_t launch_dequantize(const QuantParams &p, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const bool wide = p.cols % 8 == 0 && p.qs % 8 == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0 &&
                          reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.xs % (16 / sizeof(E)) == 0;
        const int64_t pieces = ceil_div(p.cols, 32 * kTurns * (wide ? 8 : 1)), grid = ceil_div(pieces * p.rows, 8);
        return wide ? launch_early(dequantize_kernel<E, 8>, grid, dim3(256), 0, stream, 0, p, (uint32_t)pieces)
                    : launch_early(dequantize_kernel<E, 1>, grid, dim3(256), 0, stream, 0, p, (uint32_t)pieces);
    });
}

}  // namespace kda
