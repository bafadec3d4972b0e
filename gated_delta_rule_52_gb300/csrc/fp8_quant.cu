// Quantisation to 8 bits with a power-of-two scale for each block of 128 (fp8_io.cuh), and back.
//   q = x / s,  s = 2^e for 128 neighbours of a row, or for a tile of 128 rows by 128 columns
// The transposed result has its blocks along the columns.  A CTA takes a tile of 128 x 128,
// which holds every block that it touches: the tile is read once, into registers, and both
// results come from there, the transposed one by way of shared memory.
#include <algorithm>

#include "fp8_io.cuh"
#include "layer_copy.cuh"

namespace kda {
namespace {

using namespace layer;

constexpr int kTile = kFp8Block;
constexpr int kQuantThreads = 256;

// Thread t: columns 8 (t % 16) .. + 7 of rows 64 h + 4 (t / 16) + i.
template <typename E, bool E5M2, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(QuantParams p) {
    __shared__ float tops[8][kTile];
    __shared__ float warp_top[kTile / 32];
    __shared__ uint8_t col_scale[kTile];
    __shared__ uint32_t turned[kTile * kTile / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t across = ceil_div(p.cols, kTile), br = blockIdx.x / across, bc = blockIdx.x - br * across;
    const int64_t r0 = br * kTile, c0 = bc * kTile;
    const int64_t c = c0 + 8 * cg;
    const int cols = (int)min(max(p.cols - c, (int64_t)0), (int64_t)8);
    float v[2][4][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 64 * h + 4 * rg + i;
            const E *at = static_cast<const E *>(p.x) + r * p.xs + c;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[h][i][j] = 0.f;
            if (r < p.rows) {
                constexpr int V = 16 / sizeof(E);
                if (WIDE && cols == 8) {
#pragma unroll
                    for (int j = 0; j < 8; j += V) ld_f<E, V>(at + j, reinterpret_cast<float (&)[V]>(v[h][i][j]));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < cols) v[h][i][j] = to_f(at[j]);
                }
            }
        }
    bool special = false;
    float row_top[2][4], col_top[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) col_top[j] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = finite_abs(v[h][i][j], special);
                t = fmaxf(t, a);
                col_top[j] = fmaxf(col_top[j], a);
            }
            row_top[h][i] = t;
        }
    if (p.qt || p.tile) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = fmaxf(col_top[j], __shfl_xor_sync(0xffffffffu, col_top[j], 16));
            if (lane < 16) tops[warp][8 * cg + j] = t;
        }
        __syncthreads();
        if (threadIdx.x < kTile) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) t = fmaxf(t, tops[w][threadIdx.x]);
            if (p.tile) {
#pragma unroll
                for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                if (lane == 0) warp_top[warp] = t;
            } else {
                col_scale[threadIdx.x] = (uint8_t)scale_byte(t, E5M2);
            }
        }
        __syncthreads();
    }
    int tile_scale = 0;
    if (p.tile) {
        tile_scale = scale_byte(fmaxf(fmaxf(warp_top[0], warp_top[1]), fmaxf(warp_top[2], warp_top[3])), E5M2);
        if (threadIdx.x == 0) {
            if (p.q) p.s[br * p.ss + bc] = (uint8_t)tile_scale;
            if (p.qt) p.st[bc * p.sts + br] = (uint8_t)tile_scale;
        }
    }
    if (p.q) {
        const bool whole = WIDE && cols == 8 && p.qs % 8 == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int e = tile_scale;
                if (!p.tile) {
                    float t = row_top[h][i];
#pragma unroll
                    for (int o = 8; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                    e = scale_byte(t, E5M2);
                }
                const int64_t r = r0 + 64 * h + 4 * rg + i;
                if (r >= p.rows || cols == 0) continue;
                if (!p.tile && cg == 0) p.s[r * p.ss + bc] = (uint8_t)e;
                const float inv = inverse_scale(e);
                float f[8];
                fma_n<8>(f, v[h][i], inv, 0.f);
                const uint32_t lo = quad_to_fp8<E5M2>(f[0], f[1], f[2], f[3], special), hi = quad_to_fp8<E5M2>(f[4], f[5], f[6], f[7], special);
                uint8_t *at = static_cast<uint8_t *>(p.q) + r * p.qs + c;
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
    for (int j = 0; j < 8; ++j) {
        const int col = 8 * cg + j;
        const float inv = inverse_scale(p.tile ? tile_scale : col_scale[col]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            turned[col * 32 + ((16 * h + rg + 2 * cg) & 31)] =
                quad_to_fp8<E5M2>(v[h][0][j] * inv, v[h][1][j] * inv, v[h][2][j] * inv, v[h][3][j] * inv, special);
    }
    __syncthreads();
    const bool words = p.qts % 4 == 0 && reinterpret_cast<uintptr_t>(p.qt) % 4 == 0;
    const int rows = (int)min(p.rows - r0 - 4 * lane, (int64_t)4);
    for (int col = warp; col < kTile && c0 + col < p.cols; col += 8) {
        const uint32_t w = turned[col * 32 + ((lane + 2 * (col >> 3)) & 31)];
        uint8_t *at = static_cast<uint8_t *>(p.qt) + (c0 + col) * p.qts + r0 + 4 * lane;
        if (words && rows == 4) {
            *reinterpret_cast<uint32_t *>(at) = w;
        } else {
            for (int j = 0; j < rows; ++j) at[j] = (uint8_t)(w >> (8 * j));
        }
        if (!p.tile && lane == 0) p.st[(c0 + col) * p.sts + br] = col_scale[col];
    }
}

// Scale of a byte: 2^(byte - 127), NaN for 255.  (2^-127, which is below the normal numbers,
// only where a caller wrote a 0.)
__device__ __forceinline__ float scale_of(int byte) {
    return byte == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)max(byte, 1) << 23);
}

// V neighbouring elements per thread.
template <typename E, int V>
__global__ void __launch_bounds__(256) dequantize_kernel(QuantParams p) {
    const int64_t groups = ceil_div(p.cols, V), all = groups * p.rows;
    const bool e5m2 = p.q_dtype == kE5M2;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / groups, c = (i - r * groups) * V;
        const int byte = p.s[(p.tile ? r / kTile : r) * p.ss + c / kTile];
        const float s = scale_of(byte), half = byte == 0 ? 0.5f : 1.f;
        const uint8_t *q = static_cast<const uint8_t *>(p.q) + r * p.qs + c;
        E *at = static_cast<E *>(const_cast<void *>(p.x)) + r * p.xs + c;
        if constexpr (V == 1) {
            at[0] = from_f<E>(pair_from_fp8(q[0], e5m2).x * half * s);
        } else {
            const Pack<uint32_t, V / 4> w = *reinterpret_cast<const Pack<uint32_t, V / 4> *>(q);
            float f[V];
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float2 t = pair_from_fp8(w.e[j / 4] >> (8 * (j & 2)), e5m2);
                f[j] = t.x * half * s, f[j + 1] = t.y * half * s;
            }
            constexpr int P = 16 / sizeof(E);
#pragma unroll
            for (int j = 0; j < V; j += P) st_f<E, P>(at + j, reinterpret_cast<const float (&)[P]>(f[j]));
        }
    }
}

}  // namespace

cudaError_t launch_quantize(const QuantParams &p, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const unsigned grid = (unsigned)(ceil_div(p.cols, kTile) * ceil_div(p.rows, kTile));
        const bool wide = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.xs % (16 / sizeof(E)) == 0;
        if (p.q_dtype == kE5M2) {
            if (wide) quantize_kernel<E, true, true><<<grid, kQuantThreads, 0, stream>>>(p);
            else quantize_kernel<E, true, false><<<grid, kQuantThreads, 0, stream>>>(p);
        } else {
            if (wide) quantize_kernel<E, false, true><<<grid, kQuantThreads, 0, stream>>>(p);
            else quantize_kernel<E, false, false><<<grid, kQuantThreads, 0, stream>>>(p);
        }
        return cudaGetLastError();
    });
}

cudaError_t launch_dequantize(const QuantParams &p, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const bool wide = p.cols % 16 == 0 && p.qs % 16 == 0 && reinterpret_cast<uintptr_t>(p.q) % 16 == 0 &&
                          reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.xs % (16 / sizeof(E)) == 0;
        const int64_t n = p.rows * ceil_div(p.cols, wide ? 16 : 1);
        const unsigned grid = (unsigned)std::min(ceil_div(n, 256), (int64_t)sms * 16);
        if (wide) dequantize_kernel<E, 16><<<grid, 256, 0, stream>>>(p);
        else dequantize_kernel<E, 1><<<grid, 256, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace kda
