// RMS norm over the last axis, forward and backward.
//   h = x + residual, rounded to the tensors' type;  y = h rstd w,  rstd = 1 / sqrt(mean(h^2) + eps)
//   with d = dy w, hat = h rstd:  dx = rstd (d - hat mean(d hat)) + dresidual,
//   dw = sum over rows of dy hat
// Sums are fp32.  h is rounded before it is normed, so that what the residual stream keeps is
// what the output belongs to, and the backward pass starts from it.  8-bit outputs have a scale
// for each block of 128 columns (fp8_io.cuh).
//
// A CTA takes a row; a warp takes blocks of 128 columns of it, 4 columns to a lane.
#include <algorithm>

#include "fp8_io.cuh"
#include "layer_copy.cuh"

namespace kda {
namespace {

using namespace layer;

constexpr int kRowThreads = 256;

// Sum of one value over the CTA, for all threads.
__device__ __forceinline__ float cta_sum(float v, float (&part)[32]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A lane's 4 columns of a block: neighbours where rows are aligned, else 32 apart.
template <bool WIDE>
__device__ __forceinline__ int lane_col(int lane, int j) { return WIDE ? 4 * lane + j : lane + 32 * j; }

template <typename E, bool WIDE>
__device__ __forceinline__ void ld_block(const E *p, int64_t c0, int64_t D, int lane, float (&f)[4]) {
    if (WIDE && c0 + 4 * lane + 4 <= D) {
        ld_f<E, 4>(p + c0 + 4 * lane, f);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + lane_col<WIDE>(lane, j);
        f[j] = c < D ? to_f(p[c]) : 0.f;
    }
}
template <typename E, bool WIDE>
__device__ __forceinline__ void st_block(E *p, int64_t c0, int64_t D, int lane, const float (&f)[4]) {
    if (WIDE && c0 + 4 * lane + 4 <= D) {
        st_f<E, 4>(p + c0 + 4 * lane, f);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + lane_col<WIDE>(lane, j);
        if (c < D) p[c] = from_f<E>(f[j]);
    }
}
template <bool E5M2, bool WIDE>
__device__ __forceinline__ void st_block_fp8(uint8_t *p, uint8_t *scale, int64_t c0, int64_t D, int lane, const float (&f)[4], bool words) {
    bool special = false;
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, finite_abs(f[j], special));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = scale_byte(top, E5M2);
    const float inv = inverse_scale(e);
    if (lane == 0) *scale = (uint8_t)e;
    const uint32_t w = quad_to_fp8<E5M2>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv, special);
    if (WIDE && words && c0 + 4 * lane + 4 <= D) {
        *reinterpret_cast<uint32_t *>(p + c0 + 4 * lane) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + lane_col<WIDE>(lane, j);
        if (c < D) p[c] = (uint8_t)(w >> (8 * j));
    }
}

template <typename E, bool WIDE>
__global__ void __launch_bounds__(kRowThreads) rms_fwd_kernel(RmsParams p) {
    __shared__ float part[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = kRowThreads / 32;
    const int64_t row = blockIdx.x, D = p.D, blocks = ceil_div(D, kFp8Block);
    const E *x = static_cast<const E *>(p.x) + row * p.xs;
    const E *res = p.res ? static_cast<const E *>(p.res) + row * p.rs : nullptr;
    E *sum = p.res_out ? static_cast<E *>(p.res_out) + row * p.ros : nullptr;
    float s = 0.f;
    for (int64_t b = warp; b < blocks; b += warps) {
        float h[4];
        ld_block<E, WIDE>(x, b * kFp8Block, D, lane, h);
        if (res) {
            float f[4];
            ld_block<E, WIDE>(res, b * kFp8Block, D, lane, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = to_f(from_f<E>(h[j] + f[j]));
            if (sum) st_block<E, WIDE>(sum, b * kFp8Block, D, lane, h);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(h[j], h[j], s);
    }
    const float rstd = 1.f / sqrtf(cta_sum(s, part) / (float)D + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    // The sum is read again from where this thread wrote it (it may be over x or the residual).
    const bool words = p.os % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % 4 == 0;
    for (int64_t b = warp; b < blocks; b += warps) {
        const int64_t c0 = b * kFp8Block;
        float h[4], w[4];
        ld_block<E, WIDE>(sum ? sum : x, c0, D, lane, h);
        if (res && !sum) {
            float f[4];
            ld_block<E, WIDE>(res, c0, D, lane, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = to_f(from_f<E>(h[j] + f[j]));
        }
        if (p.weight) ld_block<float, WIDE>(p.weight, c0, D, lane, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] *= p.weight ? rstd * w[j] : rstd;
        if (p.out_dtype == p.dtype) {
            st_block<E, WIDE>(static_cast<E *>(p.out) + row * p.os, c0, D, lane, h);
        } else {
            uint8_t *at = static_cast<uint8_t *>(p.out) + row * p.os, *scale = p.scales + row * p.ss + b;
            if (p.out_dtype == kE5M2) st_block_fp8<true, WIDE>(at, scale, c0, D, lane, h, words);
            else st_block_fp8<false, WIDE>(at, scale, c0, D, lane, h, words);
        }
    }
}

template <typename E, bool WIDE>
__global__ void __launch_bounds__(kRowThreads) rms_bwd_kernel(RmsParams p) {
    __shared__ float part[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = kRowThreads / 32;
    const int64_t row = blockIdx.x, D = p.D, blocks = ceil_div(D, kFp8Block);
    const E *x = static_cast<const E *>(p.x) + row * p.xs, *dy = static_cast<const E *>(p.dout) + row * p.ds;
    const E *dres = p.dres ? static_cast<const E *>(p.dres) + row * p.drs : nullptr;
    const float rstd = p.rstd[row];
    float s = 0.f;
    for (int64_t b = warp; b < blocks; b += warps) {
        float h[4], d[4], w[4];
        ld_block<E, WIDE>(x, b * kFp8Block, D, lane, h);
        ld_block<E, WIDE>(dy, b * kFp8Block, D, lane, d);
        if (p.weight) ld_block<float, WIDE>(p.weight, b * kFp8Block, D, lane, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(p.weight ? d[j] * w[j] : d[j], h[j] * rstd, s);
    }
    const float mean = cta_sum(s, part) / (float)D;
    for (int64_t b = warp; b < blocks; b += warps) {
        const int64_t c0 = b * kFp8Block;
        float h[4], d[4], w[4], f[4];
        ld_block<E, WIDE>(x, c0, D, lane, h);
        ld_block<E, WIDE>(dy, c0, D, lane, d);
        if (p.weight) ld_block<float, WIDE>(p.weight, c0, D, lane, w);
        if (dres) ld_block<E, WIDE>(dres, c0, D, lane, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float g = rstd * ((p.weight ? d[j] * w[j] : d[j]) - h[j] * rstd * mean);
            d[j] = dres ? g + f[j] : g;
        }
        st_block<E, WIDE>(static_cast<E *>(p.dx) + row * D, c0, D, lane, d);
    }
}

// Sums of dy hat over blocks of rows: a thread per column, blockIdx.y a block.
template <typename E>
__global__ void __launch_bounds__(128) rms_weight_part_kernel(RmsParams p, int64_t block_rows, float *part) {
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x, r0 = blockIdx.y * block_rows, r1 = min(r0 + block_rows, p.rows);
    if (c >= p.D) return;
    const E *x = static_cast<const E *>(p.x) + c, *dy = static_cast<const E *>(p.dout) + c;
    float s = 0.f;
#pragma unroll 4
    for (int64_t row = r0; row < r1; ++row) s = fmaf(to_f(dy[row * p.ds]), to_f(x[row * p.xs]) * p.rstd[row], s);
    part[blockIdx.y * p.D + c] = s;
}

__global__ void __launch_bounds__(kSumThreads) rms_weight_sum_kernel(RmsParams p, int64_t parts, const float *part) {
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const float t = column_sum(part, parts, p.D, c, c < p.D);
    if (threadIdx.x < 32 && c < p.D) p.dweight[c] = t;
}

// Groups of 4 elements where every row allows them.
bool wide_rows(const RmsParams &p, std::initializer_list<std::pair<const void *, int64_t>> tensors) {
    const size_t group = 4 * dtype_bytes(p.dtype);
    for (const auto &t : tensors)
        if (t.first && (reinterpret_cast<uintptr_t>(t.first) % group || t.second % 4)) return false;
    return reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;
}

int64_t weight_parts(const RmsParams &p) { return std::min(ceil_div(p.rows, 64), (int64_t)256); }

}  // namespace

size_t rms_bwd_scratch_bytes(const RmsParams &p, int) { return p.dweight ? (size_t)(weight_parts(p) * p.D) * sizeof(float) : 0; }

cudaError_t launch_rms_fwd(const RmsParams &p, int, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const bool wide = wide_rows(p, {{p.x, p.xs}, {p.res, p.rs}, {p.res_out, p.ros}}) &&
                          (p.out_dtype != p.dtype || wide_rows(p, {{p.out, p.os}}));
        if (wide) rms_fwd_kernel<E, true><<<(unsigned)p.rows, kRowThreads, 0, stream>>>(p);
        else rms_fwd_kernel<E, false><<<(unsigned)p.rows, kRowThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_rms_bwd(const RmsParams &p, unsigned char *ws, int, cudaStream_t stream) {
    float *part = reinterpret_cast<float *>(ws);
    const int64_t parts = weight_parts(p);
    const cudaError_t e = with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (p.rows == 0) return cudaSuccess;
        if (wide_rows(p, {{p.x, p.xs}, {p.dout, p.ds}, {p.dres, p.drs}, {p.dx, p.D}}))
            rms_bwd_kernel<E, true><<<(unsigned)p.rows, kRowThreads, 0, stream>>>(p);
        else rms_bwd_kernel<E, false><<<(unsigned)p.rows, kRowThreads, 0, stream>>>(p);
        if (p.dweight)
            rms_weight_part_kernel<E><<<dim3((unsigned)ceil_div(p.D, 128), (unsigned)parts), 128, 0, stream>>>(p, ceil_div(p.rows, parts), part);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !p.dweight) return e;
    rms_weight_sum_kernel<<<(unsigned)ceil_div(p.D, 32), kSumThreads, 0, stream>>>(p, parts, part);
    return cudaGetLastError();
}

}  // namespace kda
