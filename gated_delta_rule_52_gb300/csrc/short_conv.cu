// Causal depthwise short convolution, forward and backward.
//   y_t = bias + sum_j w[j] x_{t-(W-1)+j};  out = y sigma(y) (or y)
// Rows before a sequence's first are its initial state's (zero without one); the final
// state is the last W-1 rows of (initial state, sequence).
//   with q_t = dout_t act'(y_t):  dx_t = sum_k w[W-1-k] q_{t+k} (+ dfinal),
//   dw[j] = sum_t q_t x_{t-(W-1)+j}, dbias = sum_t q_t
//
// A thread walks a run of rows of V channels with its taps, its last W-1 inputs and (in the
// backward pass) its next W-1 q in registers, so a value is loaded once but for the W-1
// rows between runs.  Memory bound: 12 (forward) and 30 (backward) fp32 operations per
// element.  A row that begins a sequence replaces the inputs before it, it does not mask
// them: NaN and infinity stay within their sequence.  The weight's gradient leaves a CTA as
// one partial sum per tap and channel.
#include <algorithm>

#include "layer_copy.cuh"

namespace kda {
namespace {

using namespace layer;

constexpr int kLanes = 32, kGroups = 8, kThreads = kLanes * kGroups;

// Runs of `length` rows.  Fixed-length sequences are cut one by one (`per_seq` runs each),
// packed ones as one row range.
struct Runs { int64_t count, per_seq; int length; };

// The run of this thread: rows [r0, r1), the first one's sequence n and its rows [lo, hi).
struct Run { int64_t r0, r1, n, lo, hi; };
__device__ __forceinline__ Run run_of(const ConvParams &p, const Runs &runs, int64_t q) {
    Run r;
    if (p.cu_seqlens) {
        r.r0 = q * runs.length;
        r.r1 = min(r.r0 + runs.length, p.rows);
        r.n = seq_of_row(p.cu_seqlens, p.N, r.r0);
        seq_rows(p, r.n, r.lo, r.hi);
        r.lo = min(r.lo, r.r0);   // no row of the run lies outside, whatever cu_seqlens holds
        if (r.hi <= r.r0) r.hi = p.rows;
    } else {
        r.n = runs.per_seq == 1 ? q : q / runs.per_seq;
        r.lo = r.n * p.T;
        r.hi = r.lo + p.T;
        r.r0 = r.lo + (q - r.n * runs.per_seq) * runs.length;
        r.r1 = min(r.r0 + runs.length, r.hi);
    }
    return r;
}
// The sequence of row t = r.hi or later.
__device__ __forceinline__ void next_sequence(const ConvParams &p, Run &r, int64_t t) {
    while (r.n + 1 < p.N && r.hi <= t) seq_rows(p, ++r.n, r.lo, r.hi);
    if (r.hi <= t) r.hi = p.rows;   // rows that no sequence claims
    r.lo = t;
}

// V channels' weights, w[j][v].
template <int V, int W>
__device__ __forceinline__ void ld_taps(const float *weight, int64_t c, float (&w)[W][V]) {
    float t[V * W];
    if constexpr (V == 4) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float4 f = reinterpret_cast<const float4 *>(weight + c * W)[k];
            t[4 * k] = f.x, t[4 * k + 1] = f.y, t[4 * k + 2] = f.z, t[4 * k + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V * W; ++k) t[k] = weight[c * W + k];
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) w[j][v] = t[v * W + j];
}

// Input row t of sequence n that begins at lo, counting the initial state's rows.
template <typename E, int V>
__device__ __forceinline__ void ld_x(const ConvParams &p, int64_t n, int64_t lo, int64_t t, int64_t c, float (&f)[V]) {
    const int64_t j = t - lo + p.W - 1;
    if (t >= lo) {
        ld_f<E, V>(static_cast<const E *>(p.x) + t * p.xs + c, f);
    } else if (p.init && j >= 0) {
        ld_f<E, V>(static_cast<const E *>(p.init) + (n * (p.W - 1) + j) * p.D + c, f);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.f;
    }
}

// One step of the window: x_{t-(W-1)} .. x_t in xw; y_t.
template <int V, int W>
__device__ __forceinline__ void taps_sum(const float (&w)[W][V], const float (&b)[V], const float (&xw)[W][V], float (&y)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = b[v];
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = fmaf(w[j][v], xw[j][v], y[v]);
}
template <int V, int W>
__device__ __forceinline__ void shift(float (&xw)[W][V]) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) xw[j][v] = xw[j + 1][v];
}

template <typename E, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvParams p, Runs runs, int channel_blocks) {
    const int64_t q = (int64_t)(blockIdx.x / channel_blocks) * kGroups + threadIdx.x / kLanes;
    const int64_t c = ((int64_t)(blockIdx.x % channel_blocks) * kLanes + threadIdx.x % kLanes) * V;
    if (q >= runs.count || c >= p.D) return;
    Run r = run_of(p, runs, q);
    float w[W][V], b[V], xw[W][V];
    ld_taps<V, W>(p.weight, c, w);
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = p.bias ? p.bias[c + v] : 0.f;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) ld_x<E, V>(p, r.n, r.lo, r.r0 - (W - 1) + j, c, xw[j]);
    // the final state is the first run's to write: it alone reads the initial state
    const bool state = p.fin && !p.cu_seqlens && r.r0 == r.lo;
    float last[W - 1][V];
    if (state) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) ld_x<E, V>(p, r.n, r.lo, r.hi - (W - 1) + j, c, last[j]);
    }
    const E *x = static_cast<const E *>(p.x) + r.r0 * p.xs + c;
    E *out = static_cast<E *>(p.out) + r.r0 * p.os + c;
    constexpr int kBatch = 8;   // rows on their way together
    for (int64_t t0 = r.r0; t0 < r.r1; t0 += kBatch) {
        Pack<E, V> raw[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k, x += p.xs)
            if (t0 + k < r.r1) raw[k] = ld_pack<E, V>(x);
#pragma unroll
        for (int k = 0; k < kBatch; ++k, out += p.os) {
            const int64_t t = t0 + k;
            if (t >= r.r1) break;
            if (t == r.hi) {
                next_sequence(p, r, t);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) ld_x<E, V>(p, r.n, r.lo, t - (W - 1) + j, c, xw[j]);
            }
            unpack<E, V>(raw[k], xw[W - 1]);
            float y[V];
            taps_sum<V, W>(w, b, xw, y);
            if (p.silu) {
#pragma unroll
                for (int v = 0; v < V; ++v) y[v] *= sigmoid(y[v]);
            }
            st_f<E, V>(out, y);
            shift<V, W>(xw);
        }
    }
    if (state) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) st_f<E, V>(static_cast<E *>(p.fin) + (r.n * (W - 1) + j) * p.D + c, last[j]);
    }
}

// Final states of packed sequences (and of sequences without tokens): one thread per
// (sequence, channel), after the convolution, so that a final state may be the initial
// state's own buffer.
template <typename E>
__global__ void __launch_bounds__(kThreads) conv_state_kernel(ConvParams p) {
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= p.N * p.D) return;
    const int64_t n = at / p.D, c = at % p.D;
    int64_t lo, hi;
    seq_rows(p, n, lo, hi);
    hi = max(lo, hi);
    for (int j = 0; j < p.W - 1; ++j) {   // row j is read at or after row j: in order is safe in place
        float f[1];
        ld_x<E, 1>(p, n, lo, hi - (p.W - 1) + j, c, f);
        st_f<E, 1>(static_cast<E *>(p.fin) + (n * (p.W - 1) + j) * p.D + c, f);
    }
}

template <typename E, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvParams p, Runs runs, int channel_blocks, float *part) {
    __shared__ float sums[kGroups][W + 1][kLanes * V];
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int64_t block = blockIdx.x / channel_blocks, q = block * kGroups + group;
    const int64_t c0 = (int64_t)(blockIdx.x % channel_blocks) * kLanes * V, c = c0 + lane * V;
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    if (q < runs.count && c < p.D) {
        Run r = run_of(p, runs, q);
        float w[W][V], b[V], xw[W][V], qs[W][V];   // qs[k]: q of the row k after the current one
        ld_taps<V, W>(p.weight, c, w);
#pragma unroll
        for (int v = 0; v < V; ++v) b[v] = p.bias ? p.bias[c + v] : 0.f;

        // q of row u, whose input and upstream gradient are given; the window moves on
        const auto form_q = [&](int64_t u, const float (&x)[V], const float (&dy)[V], float (&out)[V]) {
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) xw[W - 1][v] = x[v];
            taps_sum<V, W>(w, b, xw, y);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                out[v] = dy[v];
                if (p.silu) {
                    // silu' = s + y s (1 - s) = s (1 + y (1 - s)); 1 - s as sigma(-y)
                    const float t = ex2(-kLog2e * fabsf(y[v])), rt = rcp(1.f + t), m = t * rt;
                    const float s = y[v] >= 0.f ? rt : m, o = y[v] >= 0.f ? m : rt;
                    out[v] *= s * fmaf(y[v], o, 1.f);
                }
            }
            if (u < r.r1) {   // rows after the run are another thread's to sum
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    db[v] += out[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][v] = fmaf(out[v], xw[j][v], dw[j][v]);
                }
            }
            shift<V, W>(xw);
        };
        // window and q at row t; where t begins its sequence, the initial state's gradient
        const auto start = [&](int64_t t) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) ld_x<E, V>(p, r.n, r.lo, t - (W - 1) + j, c, xw[j]);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
#pragma unroll
                for (int v = 0; v < V; ++v) qs[k][v] = 0.f;
                if (t + k < r.hi) {
                    float x[V], dy[V];
                    ld_f<E, V>(static_cast<const E *>(p.x) + (t + k) * p.xs + c, x);
                    ld_f<E, V>(static_cast<const E *>(p.dout) + (t + k) * p.ds + c, dy);
                    form_q(t + k, x, dy, qs[k]);
                }
            }
            if (t != r.lo || !p.dinit) return;
#pragma unroll
            for (int m = 0; m < W - 1; ++m) {   // state row m is input row lo - (W-1) + m
                const int64_t j = m - (r.hi - r.lo);
                float d[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[v] = p.dfinal && j >= 0 ? p.dfinal[(r.n * (W - 1) + j) * p.D + c + v] : 0.f;
#pragma unroll
                    for (int i = 0; i <= m; ++i) d[v] = fmaf(w[i][v], qs[m - i][v], d[v]);
                }
                st_f<float, V>(p.dinit + (r.n * (W - 1) + m) * p.D + c, d);
            }
        };
        start(r.r0);
        const E *x = static_cast<const E *>(p.x) + (r.r0 + W - 1) * p.xs + c;
        const E *dy = static_cast<const E *>(p.dout) + (r.r0 + W - 1) * p.ds + c;
        E *dx = static_cast<E *>(p.dx) + r.r0 * p.D + c;
        constexpr int kBatch = 4;   // rows on their way together
        for (int64_t t0 = r.r0; t0 < r.r1; t0 += kBatch) {
            Pack<E, V> rx[kBatch], rd[kBatch];   // rows W-1 ahead
#pragma unroll
            for (int k = 0; k < kBatch; ++k, x += p.xs, dy += p.ds) {
                const int64_t u = t0 + k + W - 1;
                if (t0 + k < r.r1 && u < p.rows) rx[k] = ld_pack<E, V>(x), rd[k] = ld_pack<E, V>(dy);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k, dx += p.D) {
                const int64_t t = t0 + k, u = t + W - 1;
                if (t >= r.r1) break;
                if (t == r.hi) {
                    next_sequence(p, r, t);
                    start(t);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) qs[W - 1][v] = 0.f;
                if (u < r.hi) {
                    float xf[V], df[V];
                    unpack<E, V>(rx[k], xf);
                    unpack<E, V>(rd[k], df);
                    form_q(u, xf, df, qs[W - 1]);
                }
                float d[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[v] = 0.f;
#pragma unroll
                    for (int i = 0; i < W; ++i) d[v] = fmaf(w[W - 1 - i][v], qs[i][v], d[v]);
                }
                if (p.dfinal && u >= r.hi) {
#pragma unroll
                    for (int v = 0; v < V; ++v) d[v] += p.dfinal[(r.n * (W - 1) + u - r.hi) * p.D + c + v];
                }
                st_f<E, V>(dx, d);
                shift<V, W>(qs);
            }
        }
    }
    // over the CTA's runs, in order
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) sums[group][j][lane * V + v] = dw[j][v];
        sums[group][W][lane * V + v] = db[v];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < (W + 1) * kLanes * V; k += kThreads) {
        const int j = k / (kLanes * V), l = k % (kLanes * V);
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) t += sums[g][j][l];
        if (c0 + l < p.D) part[(block * (W + 1) + j) * p.D + c0 + l] = t;
    }
}

// Sequences without tokens pass the final state's gradient to the initial state.
__global__ void __launch_bounds__(kThreads) conv_empty_kernel(ConvParams p) {
    const int64_t n = (int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes, row = (p.W - 1) * p.D;
    if (n >= p.N) return;
    int64_t lo, hi;
    seq_rows(p, n, lo, hi);
    if (lo < hi) return;
    for (int64_t k = n * row + threadIdx.x % kLanes; k < (n + 1) * row; k += kLanes) p.dinit[k] = p.dfinal ? p.dfinal[k] : 0.f;
}

// part [parts, W+1, D] to dweight [D, W] and dbias [D].
__global__ void __launch_bounds__(1024) conv_param_sum_kernel(ConvParams p, int64_t parts, const float *part) {
    const int64_t width = (p.W + 1) * p.D, k = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const float t = column_sum(part, parts, width, k, k < width);
    if (threadIdx.x >= 32 || k >= width) return;
    const int64_t j = k / p.D, c = k % p.D;
    if (j < p.W) p.dweight[c * p.W + j] = t;
    else if (p.dbias) p.dbias[c] = t;
}

// ---- host side
// 4 channels per thread where every row allows loads of 4 elements.
bool vector_rows(const ConvParams &p) {
    const size_t n = 4 * dtype_bytes(p.dtype);
    const void *ptrs[] = {p.x, p.out, p.init, p.fin, p.dout, p.dx};
    for (const void *q : ptrs)
        if (reinterpret_cast<uintptr_t>(q) % n) return false;
    if (reinterpret_cast<uintptr_t>(p.weight) % 16 || reinterpret_cast<uintptr_t>(p.dinit) % 16) return false;
    return p.D % 4 == 0 && p.xs % 4 == 0 && p.os % 4 == 0 && p.ds % 4 == 0;
}

// Runs as long as leaves about 1024 threads per SM, 8 to 64 rows: every run reads W-1 rows
// of its neighbour's again.
Runs plan_runs(const ConvParams &p, int sms) {
    const int64_t lanes = ceil_div(p.D, vector_rows(p) ? 4 : 1);
    Runs r;
    for (r.length = 64; r.length > 8 && ceil_div(p.rows, r.length) * lanes < (int64_t)sms * 1024; r.length /= 2) {}
    r.per_seq = p.cu_seqlens ? 0 : ceil_div(p.T, r.length);
    r.count = p.cu_seqlens ? ceil_div(p.rows, r.length) : p.N * r.per_seq;
    return r;
}
int64_t run_blocks(const Runs &r) { return ceil_div(r.count, kGroups); }

// Calls f(null E pointer, integral_constant V, integral_constant W).
template <typename F>
cudaError_t with_shape(const ConvParams &p, F &&f) {
    const bool vec = vector_rows(p);
    return with_dtype(p.dtype, [&](auto *tag) {
        const auto with_w = [&](auto v) {
            if (p.W == 2) return f(tag, v, std::integral_constant<int, 2>{});
            if (p.W == 3) return f(tag, v, std::integral_constant<int, 3>{});
            return f(tag, v, std::integral_constant<int, 4>{});
        };
        return vec ? with_w(std::integral_constant<int, 4>{}) : with_w(std::integral_constant<int, 1>{});
    });
}

}  // namespace

size_t conv_bwd_scratch_bytes(const ConvParams &p, int sms) {
    return (size_t)(run_blocks(plan_runs(p, sms)) * (p.W + 1) * p.D) * sizeof(float);
}

cudaError_t launch_conv_fwd(const ConvParams &p, int sms, cudaStream_t stream) {
    const Runs runs = plan_runs(p, sms);
    return with_shape(p, [&](auto *tag, auto V, auto W) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const int64_t blocks = ceil_div(p.D, kLanes * V);
        if (p.rows > 0)
            conv_fwd_kernel<E, V, W><<<(unsigned)(run_blocks(runs) * blocks), kThreads, 0, stream>>>(p, runs, (int)blocks);
        if (p.fin && (p.cu_seqlens || p.T == 0))
            conv_state_kernel<E><<<(unsigned)ceil_div(p.N * p.D, kThreads), kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_conv_bwd(const ConvParams &p, unsigned char *ws, int sms, cudaStream_t stream) {
    const Runs runs = plan_runs(p, sms);
    float *part = reinterpret_cast<float *>(ws);
    if (p.dinit && p.N > 0 && (p.cu_seqlens || p.T == 0))
        conv_empty_kernel<<<(unsigned)ceil_div(p.N, kGroups), kThreads, 0, stream>>>(p);
    const cudaError_t e = with_shape(p, [&](auto *tag, auto V, auto W) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const int64_t blocks = ceil_div(p.D, kLanes * V);
        if (p.rows > 0)
            conv_bwd_kernel<E, V, W><<<(unsigned)(run_blocks(runs) * blocks), kThreads, 0, stream>>>(p, runs, (int)blocks, part);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    conv_param_sum_kernel<<<(unsigned)ceil_div((p.W + 1) * p.D, 32), 1024, 0, stream>>>(p, run_blocks(runs), part);
    return cudaGetLastError();
}

}  // namespace kda
