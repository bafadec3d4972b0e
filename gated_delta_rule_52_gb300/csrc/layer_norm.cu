// Layer norm over the last axis, forward and backward.
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps)
//   with d = dy w, xh = (x - mean) rstd:  dx = rstd (d - mean(d) - xh mean(d xh)),
//   dw = sum over rows of dy xh, db = sum over rows of dy
// Sums are fp32; the variance is the mean square of x - mean (two passes).
//
// One CTA per row; the weight's gradient by a thread per column and row block.
#include "layer_io.cuh"

namespace kda {
namespace {

using namespace layer;

constexpr int kThreads = 256;

__device__ float block_sum(float v) {
    __shared__ float part[kThreads / 32];
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) v += part[w];
    return v;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(NormParams p) {
    const int64_t row = blockIdx.x;
    const E *x = static_cast<const E *>(p.x) + row * p.xs;
    E *out = static_cast<E *>(p.out) + row * p.os;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) s += to_f(x[c]);
    const float mean = block_sum(s) / (float)p.D;
    s = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) {
        const float d = to_f(x[c]) - mean;
        s += d * d;
    }
    const float rstd = 1.f / sqrtf(block_sum(s) / (float)p.D + p.eps);
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) {
        const float xh = (to_f(x[c]) - mean) * rstd;
        out[c] = from_f<E>(xh * (p.weight ? p.weight[c] : 1.f) + (p.bias ? p.bias[c] : 0.f));
    }
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(NormParams p) {
    const int64_t row = blockIdx.x;
    const E *x = static_cast<const E *>(p.x) + row * p.xs, *dy = static_cast<const E *>(p.dout) + row * p.ds;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) {
        const float d = to_f(dy[c]) * (p.weight ? p.weight[c] : 1.f);
        s1 += d;
        s2 += d * ((to_f(x[c]) - mean) * rstd);
    }
    s1 = block_sum(s1) / (float)p.D;
    s2 = block_sum(s2) / (float)p.D;
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) {
        const float d = to_f(dy[c]) * (p.weight ? p.weight[c] : 1.f), xh = (to_f(x[c]) - mean) * rstd;
        static_cast<E *>(p.dx)[row * p.D + c] = from_f<E>(rstd * (d - s1 - xh * s2));
    }
}

// Rows per partial sum of the weight's gradient.
constexpr int64_t kPartRows = 128;

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_param_part_kernel(NormParams p, float *dw, float *db) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x, r0 = blockIdx.y * kPartRows;
    if (c >= p.D) return;
    float w = 0.f, b = 0.f;
    for (int64_t row = r0; row < min(r0 + kPartRows, p.rows); ++row) {
        const float dy = to_f(static_cast<const E *>(p.dout)[row * p.ds + c]);
        w += dy * ((to_f(static_cast<const E *>(p.x)[row * p.xs + c]) - p.mean[row]) * p.rstd[row]);
        b += dy;
    }
    dw[blockIdx.y * p.D + c] = w;
    db[blockIdx.y * p.D + c] = b;
}

__global__ void __launch_bounds__(kThreads) norm_param_sum_kernel(NormParams p, int64_t parts, const float *dw,
                                                                  const float *db) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= p.D) return;
    float w = 0.f, b = 0.f;
    for (int64_t j = 0; j < parts; ++j) {
        w += dw[j * p.D + c];
        b += db[j * p.D + c];
    }
    if (p.dweight) p.dweight[c] = w;
    if (p.dbias) p.dbias[c] = b;
}

// Partial sums: at most 65535 (a grid's y extent), so the rows of a launch are bounded.
int64_t norm_parts(const NormParams &p) { return ceil_div(p.rows, kPartRows); }

}  // namespace

size_t norm_bwd_scratch_bytes(const NormParams &p, int) {
    return p.dweight || p.dbias ? (size_t)(2 * norm_parts(p) * p.D) * sizeof(float) : 0;
}

cudaError_t launch_norm_fwd(const NormParams &p, int, cudaStream_t stream) {
    with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        norm_fwd_kernel<E><<<(unsigned)p.rows, kThreads, 0, stream>>>(p);
    });
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormParams &p, unsigned char *ws, int, cudaStream_t stream) {
    const int64_t parts = norm_parts(p);
    const unsigned cols = (unsigned)ceil_div(p.D, kThreads);
    float *dw = reinterpret_cast<float *>(ws), *db = dw + parts * p.D;
    with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (p.rows > 0) norm_bwd_kernel<E><<<(unsigned)p.rows, kThreads, 0, stream>>>(p);
        if ((p.dweight || p.dbias) && p.rows > 0)
            norm_param_part_kernel<E><<<dim3(cols, (unsigned)parts), kThreads, 0, stream>>>(p, dw, db);
    });
    if (p.dweight || p.dbias) norm_param_sum_kernel<<<cols, kThreads, 0, stream>>>(p, parts, dw, db);
    return cudaGetLastError();
}

}  // namespace kda
