// Causal depthwise short convolution, forward and backward.
//   y_t = bias + sum_j w[j] x_{t-(W-1)+j};  out = y sigma(y) (or y)
// Rows before a sequence's first are its initial state's (zero without one); the final
// state is the last W-1 rows of (initial state, sequence).
//   with q_t = dout_t act'(y_t):  dx_t = sum_j w[j] q_{t+(W-1)-j} (+ dfinal),
//   dw[j] = sum_t q_t x_{t-(W-1)+j}, dbias = sum_t q_t
//
// One thread per (row, channel).
#include "layer_io.cuh"

namespace kda {
namespace {

using namespace layer;

constexpr int kThreads = 256;

// The sequence of a packed row and its rows [lo, hi).
__device__ __forceinline__ int64_t conv_seq(const ConvParams &p, int64_t row, int64_t &lo, int64_t &hi) {
    const int64_t n = p.cu_seqlens ? seq_of_row(p.cu_seqlens, p.N, row) : row / p.T;
    seq_rows(p, n, lo, hi);
    return n;
}

// Input row r of sequence n (rows [lo, ...)), counting the state's rows before lo.
template <typename E>
__device__ __forceinline__ float conv_x(const ConvParams &p, int64_t n, int64_t lo, int64_t r, int64_t c) {
    if (r >= lo) return to_f(static_cast<const E *>(p.x)[r * p.xs + c]);
    const int64_t j = r - lo + p.W - 1;
    return p.init && j >= 0 ? to_f(static_cast<const E *>(p.init)[(n * (p.W - 1) + j) * p.D + c]) : 0.f;
}

template <typename E>
__device__ float conv_y(const ConvParams &p, int64_t n, int64_t lo, int64_t r, int64_t c) {
    float y = p.bias ? p.bias[c] : 0.f;
    for (int j = 0; j < p.W; ++j) y += p.weight[c * p.W + j] * conv_x<E>(p, n, lo, r - (p.W - 1) + j, c);
    return y;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvParams p) {
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= p.rows * p.D) return;
    const int64_t row = at / p.D, c = at % p.D;
    int64_t lo, hi;
    const int64_t n = conv_seq(p, row, lo, hi);
    const float y = conv_y<E>(p, n, lo, row, c);
    static_cast<E *>(p.out)[row * p.os + c] = from_f<E>(p.silu ? y * sigmoid(y) : y);
}

// Final states: one thread per (sequence, channel), so that a final state may be the
// initial state's own buffer.
template <typename E>
__global__ void __launch_bounds__(kThreads) conv_state_kernel(ConvParams p) {
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= p.N * p.D) return;
    const int64_t n = at / p.D, c = at % p.D;
    int64_t lo, hi;
    seq_rows(p, n, lo, hi);
    hi = max(lo, hi);
    for (int j = 0; j < p.W - 1; ++j)   // row j is read at or after row j: in order is safe in place
        static_cast<E *>(p.fin)[(n * (p.W - 1) + j) * p.D + c] = from_f<E>(conv_x<E>(p, n, lo, hi - (p.W - 1) + j, c));
}

template <typename E>
__device__ float conv_q(const ConvParams &p, int64_t n, int64_t lo, int64_t r, int64_t c) {
    const float dy = to_f(static_cast<const E *>(p.dout)[r * p.ds + c]);
    if (!p.silu) return dy;
    const float y = conv_y<E>(p, n, lo, r, c);
    float s, slope;
    sigmoid_slope(y, s, slope);
    return dy * (s + y * slope);
}

template <typename E>
__global__ void __launch_bounds__(kThreads) conv_dx_kernel(ConvParams p) {
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= p.rows * p.D) return;
    const int64_t row = at / p.D, c = at % p.D;
    int64_t lo, hi;
    const int64_t n = conv_seq(p, row, lo, hi);
    float d = 0.f;
    for (int j = 0; j < p.W; ++j) {
        const int64_t r = row + (p.W - 1) - j;
        if (r < hi) d += p.weight[c * p.W + j] * conv_q<E>(p, n, lo, r, c);
    }
    const int64_t j = row - hi + p.W - 1;
    if (p.dfinal && j >= 0) d += p.dfinal[(n * (p.W - 1) + j) * p.D + c];
    static_cast<E *>(p.dx)[row * p.D + c] = from_f<E>(d);
}

template <typename E>
__global__ void __launch_bounds__(kThreads) conv_dinit_kernel(ConvParams p) {
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= p.N * p.D) return;
    const int64_t n = at / p.D, c = at % p.D;
    int64_t lo, hi;
    seq_rows(p, n, lo, hi);
    hi = max(lo, hi);
    for (int m = 0; m < p.W - 1; ++m) {   // state row m is input row lo - (W-1) + m
        float d = 0.f;
        for (int j = 0; j <= m; ++j) {
            const int64_t r = lo + m - j;
            if (r < hi) d += p.weight[c * p.W + j] * conv_q<E>(p, n, lo, r, c);
        }
        const int64_t j = m - (hi - lo);
        if (p.dfinal && j >= 0) d += p.dfinal[(n * (p.W - 1) + j) * p.D + c];
        p.dinit[(n * (p.W - 1) + m) * p.D + c] = d;
    }
}

constexpr int64_t kPartRows = 128;

// Partial sums [parts, W+1, D] of the weight's and the bias's gradient.
template <typename E>
__global__ void __launch_bounds__(kThreads) conv_param_part_kernel(ConvParams p, float *part) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x, r0 = blockIdx.y * kPartRows;
    if (c >= p.D) return;
    float dw[4] = {}, db = 0.f;
    for (int64_t row = r0; row < min(r0 + kPartRows, p.rows); ++row) {
        int64_t lo, hi;
        const int64_t n = conv_seq(p, row, lo, hi);
        const float q = conv_q<E>(p, n, lo, row, c);
        for (int j = 0; j < 4; ++j)
            if (j < p.W) dw[j] += q * conv_x<E>(p, n, lo, row - (p.W - 1) + j, c);
        db += q;
    }
    for (int j = 0; j < 4; ++j)
        if (j < p.W) part[((int64_t)blockIdx.y * (p.W + 1) + j) * p.D + c] = dw[j];
    part[((int64_t)blockIdx.y * (p.W + 1) + p.W) * p.D + c] = db;
}

__global__ void __launch_bounds__(kThreads) conv_param_sum_kernel(ConvParams p, int64_t parts, const float *part) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= p.D) return;
    for (int j = 0; j <= p.W; ++j) {
        float s = 0.f;
        for (int64_t k = 0; k < parts; ++k) s += part[(k * (p.W + 1) + j) * p.D + c];
        if (j < p.W) p.dweight[c * p.W + j] = s;
        else if (p.dbias) p.dbias[c] = s;
    }
}

}  // namespace

size_t conv_bwd_scratch_bytes(const ConvParams &p, int) {
    return (size_t)(ceil_div(p.rows, kPartRows) * (p.W + 1) * p.D) * sizeof(float);
}

cudaError_t launch_conv_fwd(const ConvParams &p, int, cudaStream_t stream) {
    with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (p.rows > 0) conv_fwd_kernel<E><<<(unsigned)ceil_div(p.rows * p.D, kThreads), kThreads, 0, stream>>>(p);
        if (p.fin) conv_state_kernel<E><<<(unsigned)ceil_div(p.N * p.D, kThreads), kThreads, 0, stream>>>(p);
    });
    return cudaGetLastError();
}

cudaError_t launch_conv_bwd(const ConvParams &p, unsigned char *ws, int, cudaStream_t stream) {
    const int64_t parts = ceil_div(p.rows, kPartRows);
    const unsigned cols = (unsigned)ceil_div(p.D, kThreads);
    float *part = reinterpret_cast<float *>(ws);
    with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (p.rows > 0) {
            conv_dx_kernel<E><<<(unsigned)ceil_div(p.rows * p.D, kThreads), kThreads, 0, stream>>>(p);
            conv_param_part_kernel<E><<<dim3(cols, (unsigned)parts), kThreads, 0, stream>>>(p, part);
        }
        if (p.dinit && p.N > 0) conv_dinit_kernel<E><<<(unsigned)ceil_div(p.N * p.D, kThreads), kThreads, 0, stream>>>(p);
    });
    conv_param_sum_kernel<<<cols, kThreads, 0, stream>>>(p, parts, part);
    return cudaGetLastError();
}

}  // namespace kda
