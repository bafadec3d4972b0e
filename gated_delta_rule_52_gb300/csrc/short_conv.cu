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

// Rows [r0, r1) of a thread's run, and the part [s0, s1) of them that lies in sequence n,
// whose rows are [lo, hi).
struct Run { int64_t r0, r1, s0, s1, n, lo, hi; };
__device__ __forceinline__ void part_of_run(const ConvParams &p, Run &r) {
    r.lo = min(r.lo, r.s0);   // no row of the run lies outside, whatever cu_seqlens holds
    if (r.hi <= r.s0) r.hi = p.rows;
    r.s1 = min(r.r1, r.hi);
}
__device__ __forceinline__ Run run_of(const ConvParams &p, const Runs &runs, int64_t q) {
    Run r;
    if (p.cu_seqlens) {
        r.r0 = q * runs.length;
        r.r1 = min(r.r0 + runs.length, p.rows);
        r.n = seq_of_row(p.cu_seqlens, p.N, r.r0);
        seq_rows(p, r.n, r.lo, r.hi);
    } else {
        r.n = runs.per_seq == 1 ? q : q / runs.per_seq;
        r.lo = r.n * p.T;
        r.hi = r.lo + p.T;
        r.r0 = r.lo + (q - r.n * runs.per_seq) * runs.length;
        r.r1 = min(r.r0 + runs.length, r.hi);
    }
    r.s0 = r.r0;
    part_of_run(p, r);
    return r;
}
// The part of the run in the next sequence that has rows; false at the run's end.
__device__ __forceinline__ bool next_part(const ConvParams &p, Run &r) {
    if (r.s1 >= r.r1) return false;
    r.s0 = r.s1;
    while (r.n + 1 < p.N && r.hi <= r.s0) seq_rows(p, ++r.n, r.lo, r.hi);
    part_of_run(p, r);
    return true;
}

// V channels per thread.  WIDE: every row allows loads of V elements; else they are moved
// one by one, and a thread's last channels may not exist.
constexpr int V = 4;

// A thread's weights, w[j][v].
template <bool WIDE, int W>
__device__ __forceinline__ void ld_taps(const float *weight, int64_t c, int cols, float (&w)[W][V]) {
    float t[V * W];
    if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float4 f = reinterpret_cast<const float4 *>(weight + c * W)[k];
            t[4 * k] = f.x, t[4 * k + 1] = f.y, t[4 * k + 2] = f.z, t[4 * k + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V * W; ++k) t[k] = k < cols * W ? weight[c * W + k] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) w[j][v] = t[v * W + j];
}

// Input row t of sequence n that begins at lo, counting the initial state's rows.
template <typename E, int V, bool WIDE>
__device__ __forceinline__ void ld_x(const ConvParams &p, int64_t n, int64_t lo, int64_t t, int64_t c, int cols, float (&f)[V]) {
    const int64_t j = t - lo + p.W - 1;
    if (t >= lo) {
        ld_cols<E, V, WIDE>(static_cast<const E *>(p.x) + t * p.xs + c, f, cols);
    } else if (p.init && j >= 0) {
        ld_cols<E, V, WIDE>(static_cast<const E *>(p.init) + (n * (p.W - 1) + j) * p.D + c, f, cols);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.f;
    }
}

// y_t of the window x_{t-(W-1)} .. x_t.
template <int W>
__device__ __forceinline__ void taps_sum(const float (&w)[W][V], const float (&b)[V], const float (&xw)[W][V], float (&y)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = b[v];
#pragma unroll
    for (int j = 0; j < W; ++j) fma_n<V>(y, w[j], xw[j], y);
}
template <int W>
__device__ __forceinline__ void shift(float (&xw)[W][V]) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) xw[j][v] = xw[j + 1][v];
}

// Calls f with every state element of the packed sequences without tokens, which no run
// comes to: sequence n is CTA n's.
template <typename F>
__device__ __forceinline__ void each_empty(const ConvParams &p, F &&f) {
    for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
        int64_t lo, hi;
        seq_rows(p, n, lo, hi);
        if (lo < hi) continue;
        const int64_t size = (p.W - 1) * p.D;
        for (int64_t k = n * size + threadIdx.x; k < (n + 1) * size; k += blockDim.x) f(k);
    }
}

constexpr int kBatch = 4, kStages = 3;   // rows per copy group, groups of a thread's ring

// 16384 x 4096 fp16, W = 4: 56 us, 4.8 TB/s, issue at 62% (a plain copy of the same bytes
// 47 us).
template <typename E, bool WIDE, int W>
__global__ void __launch_bounds__(kThreads, 4) conv_fwd_kernel(ConvParams p, Runs runs, int channel_blocks) {
    extern __shared__ __align__(16) unsigned char smem[];
    auto &ring = *reinterpret_cast<RowSlot<E, V, WIDE>(*)[kStages][kBatch][kThreads]>(smem);
    const int tid = threadIdx.x;
    const int64_t q = (int64_t)(blockIdx.x / channel_blocks) * kGroups + tid / kLanes;
    const int64_t c = ((int64_t)(blockIdx.x % channel_blocks) * kLanes + tid % kLanes) * V;
    const int cols = (int)min(p.D - c, (int64_t)V);
    if (p.cu_seqlens && p.fin)
        each_empty(p, [&](int64_t k) { static_cast<E *>(p.fin)[k] = p.init ? static_cast<const E *>(p.init)[k] : from_f<E>(0.f); });
    if (q >= runs.count || cols <= 0) return;
    Run r = run_of(p, runs, q);
    float w[W][V], b[V], xw[W][V];
    ld_taps<WIDE, W>(p.weight, c, cols, w);
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = p.bias && v < cols ? p.bias[c + v] : 0.f;
    do {
        const int own = (int)(r.s1 - r.s0);
        const auto fetch = [&](int j0, int stage) {
            copy_rows<E, V, WIDE, kBatch, kThreads>(&ring[stage][0][tid], static_cast<const E *>(p.x) + (r.s0 + j0) * p.xs + c, p.xs, own - j0, cols);
            copies_commit();
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) fetch(k * kBatch, k);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) ld_x<E, V, WIDE>(p, r.n, r.lo, r.s0 - (W - 1) + j, c, cols, xw[j]);
        E *out = static_cast<E *>(p.out) + r.s0 * p.os + c;
        const RowParity odd(static_cast<const E *>(p.x) + r.s0 * p.xs + c, p.xs);   // batches begin at even rows
        const auto row = [&](int k, int stage) {
            take<E, V>(ring[stage][k][tid], odd[k], xw[W - 1]);
            float y[V], s[V];
            taps_sum<W>(w, b, xw, y);
            if (p.silu) {
                sigmoid_n<V>(s, y);
                mul_n<V>(y, y, s);
            }
            st_cols<E, V, WIDE>(out, y, cols);
            out += p.os;
            shift<W>(xw);
        };
        for (int j0 = 0, stage = 0; j0 < own; j0 += kBatch) {
            fetch(j0 + (kStages - 1) * kBatch, stage == 0 ? kStages - 1 : stage - 1);
            copies_wait<kStages - 1>();   // this thread's own copies: no barrier needed
            if (j0 + kBatch <= own) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k) row(k, stage);
            } else {
#pragma unroll 1
                for (int k = 0; k < own - j0; ++k) row(k, stage);
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        // the window after a sequence's last row is its final state
        if (p.fin && r.s1 == r.hi) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) st_cols<E, V, WIDE>(static_cast<E *>(p.fin) + (r.n * (W - 1) + j) * p.D + c, xw[j], cols);
        }
    } while (next_part(p, r));
    copies_wait<0>();
}

// Final states of calls whose final state is the initial state's own buffer, which several
// runs read: one thread per (sequence, channel), after the convolution.
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
        ld_x<E, 1, true>(p, n, lo, hi - (p.W - 1) + j, c, 1, f);
        st_f<E, 1>(static_cast<E *>(p.fin) + (n * (p.W - 1) + j) * p.D + c, f);
    }
}

// With t = u - (W-1), row u's q completes d_t = sum_k w[W-1-k] q_{t+k}: the gradient of
// input row t, or of a row of the initial state where t comes before the sequence.  So a
// part [s0, s1) of a run walks u from s0 to s1 + W-2; rows from s1 on add to no parameter,
// and rows after the sequence have a q of 0 but the final state's gradient.
// 8192 x 8192 bf16, W = 4: 100 us, 4.0 TB/s; bound by issue and dependent arithmetic at the
// 16 warps per SM that its windows' registers leave.  2 channels per thread: 123 us; a ring
// filled by tensor maps: 102 us, and the forward pass's call of one token 16 us instead of 9.
template <typename E, bool WIDE, int W>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(ConvParams p, Runs runs, int channel_blocks, float *part) {
    extern __shared__ __align__(16) unsigned char smem[];
    auto &ring = *reinterpret_cast<RowSlot<E, V, WIDE>(*)[kStages][2][kBatch][kThreads]>(smem);   // x, dout
    auto &sums = *reinterpret_cast<float (*)[kGroups][W + 1][kLanes * V]>(smem);         // after the walk
    const int tid = threadIdx.x, lane = tid % kLanes, group = tid / kLanes;
    const int64_t block = blockIdx.x / channel_blocks, q = block * kGroups + group;
    const int64_t c0 = (int64_t)(blockIdx.x % channel_blocks) * kLanes * V, c = c0 + lane * V;
    // a sequence without tokens passes the final state's gradient to the initial state
    if (p.cu_seqlens && p.dinit) each_empty(p, [&](int64_t k) { p.dinit[k] = p.dfinal ? p.dfinal[k] : 0.f; });
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    const int cols = (int)min(p.D - c, (int64_t)V);
    if (q < runs.count && cols > 0) {
        Run r = run_of(p, runs, q);
        float w[W][V], b[V];
        ld_taps<WIDE, W>(p.weight, c, cols, w);
#pragma unroll
        for (int v = 0; v < V; ++v) b[v] = p.bias && v < cols ? p.bias[c + v] : 0.f;
        do {
            const int own = (int)(r.s1 - r.s0), real = own + (int)min((int64_t)(W - 1), r.hi - r.s1), all = own + W - 1;
            const bool first = r.s0 == r.lo;
            const auto fetch = [&](int j0, int stage) {
                const E *x = static_cast<const E *>(p.x) + (r.s0 + j0) * p.xs + c, *dy = static_cast<const E *>(p.dout) + (r.s0 + j0) * p.ds + c;
                copy_rows<E, V, WIDE, kBatch, kThreads>(&ring[stage][0][0][tid], x, p.xs, real - j0, cols);
                copy_rows<E, V, WIDE, kBatch, kThreads>(&ring[stage][1][0][tid], dy, p.ds, real - j0, cols);
                copies_commit();
            };
            float xw[W][V], qs[W][V];   // inputs u-(W-1) .. u and their q
#pragma unroll
            for (int k = 0; k < kStages - 1; ++k) fetch(k * kBatch, k);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                ld_x<E, V, WIDE>(p, r.n, r.lo, r.s0 - (W - 1) + j, c, cols, xw[j]);
#pragma unroll
                for (int v = 0; v < V; ++v) qs[j][v] = 0.f;
            }
            E *dx = static_cast<E *>(p.dx) + (r.s0 - (W - 1)) * p.D + c;
            const RowParity x_odd(static_cast<const E *>(p.x) + r.s0 * p.xs + c, p.xs), d_odd(static_cast<const E *>(p.dout) + r.s0 * p.ds + c, p.ds);
            // q of the row in slot k, whose window is complete
            const auto form_q = [&](int k, int stage) {
                float (&qn)[V] = qs[W - 1];
                take<E, V>(ring[stage][0][k][tid], x_odd[k], xw[W - 1]);
                take<E, V>(ring[stage][1][k][tid], d_odd[k], qn);
                if (p.silu) {   // silu' = s (1 + y (1 - s))
                    float y[V], s[V], o[V], one[V];
                    taps_sum<W>(w, b, xw, y);
                    sigmoid_n<V>(s, y);
                    fma_n<V>(o, s, -1.f, 1.f);
#pragma unroll
                    for (int v = 0; v < V; ++v) one[v] = 1.f;
                    fma_n<V>(o, y, o, one);
                    mul_n<V>(s, s, o);
                    mul_n<V>(qn, qn, s);
                }
            };
            const auto add_params = [&]() {
                add_n<V>(db, db, qs[W - 1]);
#pragma unroll
                for (int i = 0; i < W; ++i) fma_n<V>(dw[i], qs[W - 1], xw[i], dw[i]);
            };
            const auto form_d = [&](float (&d)[V]) {
                mul_n<V>(d, w[W - 1], qs[0]);
#pragma unroll
                for (int i = 1; i < W; ++i) fma_n<V>(d, w[W - 1 - i], qs[i], d);
            };
            for (int j0 = 0, stage = 0; j0 < all; j0 += kBatch) {
                fetch(j0 + (kStages - 1) * kBatch, stage == 0 ? kStages - 1 : stage - 1);
                copies_wait<kStages - 1>();   // this thread's own copies: no barrier needed
                if (j0 >= W - 1 && j0 + kBatch <= own) {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k, dx += p.D) {
                        float d[V];
                        form_q(k, stage);
                        add_params();
                        form_d(d);
                        st_cols<E, V, WIDE>(dx, d, cols);
                        shift<W>(xw);
                        shift<W>(qs);
                    }
                } else {
                    // the part's first and last rows
                    const int n = min(kBatch, all - j0);
#pragma unroll 1
                    for (int k = 0; k < n; ++k, dx += p.D) {
                        const int j = j0 + k;
                        if (j < real) {
                            form_q(k, stage);
                            if (j < own) add_params();
                        } else {
#pragma unroll
                            for (int v = 0; v < V; ++v) qs[W - 1][v] = 0.f;
                        }
                        float d[V];
                        form_d(d);
                        if (p.dfinal && r.s0 + j >= r.hi) {
#pragma unroll
                            for (int v = 0; v < V; ++v)
                                if (v < cols) d[v] += p.dfinal[(r.n * (W - 1) + (r.s0 + j - r.hi)) * p.D + c + v];
                        }
                        if (j >= W - 1) st_cols<E, V, WIDE>(dx, d, cols);
                        else if (first && p.dinit) st_cols<float, V, WIDE>(p.dinit + (r.n * (W - 1) + j) * p.D + c, d, cols);
                        shift<W>(xw);
                        shift<W>(qs);
                    }
                }
                stage = stage + 1 == kStages ? 0 : stage + 1;
            }
        } while (next_part(p, r));
    }
    copies_wait<0>();
    __syncthreads();
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

// The same for a call without any token.
__global__ void __launch_bounds__(kThreads) conv_empty_kernel(ConvParams p) {
    each_empty(p, [&](int64_t k) { p.dinit[k] = p.dfinal ? p.dfinal[k] : 0.f; });
}

// part [parts, W+1, D] to dweight [D, W] and dbias [D].
__global__ void __launch_bounds__(kSumThreads) conv_param_sum_kernel(ConvParams p, int64_t parts, const float *part) {
    const int64_t width = (p.W + 1) * p.D, k = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const float t = column_sum(part, parts, width, k, k < width);
    if (threadIdx.x >= 32 || k >= width) return;
    const int64_t j = k / p.D, c = k % p.D;
    if (j < p.W) p.dweight[c * p.W + j] = t;
    else if (p.dbias) p.dbias[c] = t;
}

// ---- host side
// Whether every row allows loads of 4 elements.
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
    const int64_t lanes = ceil_div(p.D, V);
    Runs r;
    for (r.length = 64; r.length > 8 && ceil_div(p.rows, r.length) * lanes < (int64_t)sms * 1024; r.length /= 2) {}
    r.per_seq = p.cu_seqlens ? 0 : ceil_div(p.T, r.length);
    r.count = p.cu_seqlens ? ceil_div(p.rows, r.length) : p.N * r.per_seq;
    return r;
}
int64_t run_blocks(const Runs &r) { return ceil_div(r.count, kGroups); }

// Calls f(null E pointer, bool_constant WIDE, integral_constant W).
template <typename F>
cudaError_t with_shape(const ConvParams &p, F &&f) {
    const bool wide = vector_rows(p);
    return with_dtype(p.dtype, [&](auto *tag) {
        const auto with_w = [&](auto v) {
            if (p.W == 2) return f(tag, v, std::integral_constant<int, 2>{});
            if (p.W == 3) return f(tag, v, std::integral_constant<int, 3>{});
            return f(tag, v, std::integral_constant<int, 4>{});
        };
        return wide ? with_w(std::true_type{}) : with_w(std::false_type{});
    });
}

}  // namespace

size_t conv_bwd_scratch_bytes(const ConvParams &p, int sms) {
    return (size_t)(run_blocks(plan_runs(p, sms)) * (p.W + 1) * p.D) * sizeof(float);
}

cudaError_t launch_conv_fwd(const ConvParams &p0, int sms, cudaStream_t stream) {
    ConvParams p = p0;
    const Runs runs = plan_runs(p, sms);
    // the convolution writes the final states unless it may still read them as initial ones
    const bool apart = p.fin && (p.rows == 0 || (p.fin == p.init && (p.cu_seqlens || runs.per_seq > 1)));
    if (apart) p.fin = nullptr;
    return with_shape(p0, [&](auto *tag, auto WIDE, auto W) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const int64_t blocks = ceil_div(p.D, kLanes * V);
        if (p.rows > 0) {
            constexpr auto kernel = conv_fwd_kernel<E, WIDE, W>;
            constexpr int smem = (int)sizeof(RowSlot<E, V, WIDE>) * kStages * kBatch * kThreads;
            const cudaError_t e = allow_smem<kernel>(smem);
            if (e != cudaSuccess) return e;
            kernel<<<(unsigned)(run_blocks(runs) * blocks), kThreads, smem, stream>>>(p, runs, (int)blocks);
        }
        if (apart) conv_state_kernel<E><<<(unsigned)ceil_div(p.N * p.D, kThreads), kThreads, 0, stream>>>(p0);
        return cudaGetLastError();
    });
}

cudaError_t launch_conv_bwd(const ConvParams &p, unsigned char *ws, int sms, cudaStream_t stream) {
    const Runs runs = plan_runs(p, sms);
    float *part = reinterpret_cast<float *>(ws);
    if (p.rows == 0 && p.dinit && p.N > 0)
        conv_empty_kernel<<<(unsigned)std::min(p.N, (int64_t)sms), kThreads, 0, stream>>>(p);
    const cudaError_t e = with_shape(p, [&](auto *tag, auto WIDE, auto W) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const int64_t blocks = ceil_div(p.D, kLanes * V);
        if (p.rows == 0) return cudaSuccess;
        constexpr auto kernel = conv_bwd_kernel<E, WIDE, W>;
        constexpr int smem = (int)std::max(sizeof(RowSlot<E, V, WIDE>) * kStages * 2 * kBatch * kThreads, sizeof(float) * kGroups * (W + 1) * kLanes * V);
        const cudaError_t e = allow_smem<kernel>(smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)(run_blocks(runs) * blocks), kThreads, smem, stream>>>(p, runs, (int)blocks, part);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    conv_param_sum_kernel<<<(unsigned)ceil_div((p.W + 1) * p.D, 32), kSumThreads, 0, stream>>>(p, run_blocks(runs), part);
    return cudaGetLastError();
}

}  // namespace kda
