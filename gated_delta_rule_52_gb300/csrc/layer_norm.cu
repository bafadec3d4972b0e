// Layer norm over the last axis, forward and backward.
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps)
//   with d = dy w, xh = (x - mean) rstd:  dx = rstd (d - mean(d) - xh mean(d xh)),
//   dw = sum over rows of dy xh, db = sum over rows of dy
// Sums are fp32; the variance is the mean square of x - mean, formed after the mean from
// the row that the threads hold in registers.
//
// Both directions move each value once.  Threads blockDim.x share a row (a warp for short
// rows, then blockDim.y rows per CTA), EL elements each.  The backward kernel is
// persistent: a CTA walks its rows with the next ones on their way into shared memory, a
// thread keeps its columns' weights and their gradients in registers, and one partial sum
// per CTA and column is left for a second kernel.  The forward kernel for many 16-bit rows
// walks them likewise.  Rows too long for registers (more than 16384 forward; backward 8192,
// or 4096 unaligned in 16 bits) run kernels that pass over a row again through L2.
#include <algorithm>

#include "layer_copy.cuh"

namespace kda {
namespace {

using namespace layer;

constexpr int kMaxWarps = 32;

// Sum of one value over the blockDim.x threads of every row of the CTA; all threads of the
// CTA call it together.  `part`: one warp's sum each; a caller's next call must use another.
__device__ __forceinline__ float row_sum(float v, float (&part)[kMaxWarps]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    const int first = threadIdx.y * warps, lane = threadIdx.x & 31;
    if (lane == 0) part[first + (threadIdx.x >> 5)] = v;
    __syncthreads();
    v = lane < warps ? part[first + lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The same for two values, at most 16 warps per row: one half of the lanes sums a, the
// other b, half the shuffles of two sums.
__device__ __forceinline__ void row_sum2(float &a, float &b, float (&part)[2][kMaxWarps]) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool low = lane < 16;
    float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps > 1) {
        const int first = threadIdx.y * warps, k = lane >> 4, l = lane & 15;
        if (l == 0) part[k][first + (threadIdx.x >> 5)] = v;
        __syncthreads();
        v = l < warps ? part[k][first + l] : 0.f;
#pragma unroll
        for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}
template <int n>
__device__ __forceinline__ float lane_sum(const float (&v)[n]) {
    float t[2] = {0.f, 0.f};
    if constexpr (n % 2 == 0) {
#pragma unroll
        for (int j = 0; j < n; j += 2) add_n<2>(t, t, reinterpret_cast<const float (&)[2]>(v[j]));
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j) t[0] += v[j];
    }
    return t[0] + t[1];
}

// Column of group k of a thread: groups of V, neighbouring threads side by side.
template <int V>
__device__ __forceinline__ int column(int k) { return (k * blockDim.x + threadIdx.x) * V; }

template <int V>
__device__ __forceinline__ void ld_param(const float *p, int c, float dflt, float (&f)[V]) {
    if (!p) {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = dflt;
        return;
    }
    if constexpr (V >= 4) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(p + c + v);
            f[v] = t.x, f[v + 1] = t.y, f[v + 2] = t.z, f[v + 3] = t.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = p[c + v];
    }
}

// A row per CTA, or a warp to a short one.  Bound by latency: a row's loads, two sums over
// its threads and its stores follow each other.  8192 x 8192 in 32 bits: 84 us, 6.4 TB/s.
template <typename E, int V, int EL>
__global__ void __launch_bounds__(EL == 32 ? 512 : 1024) norm_fwd_kernel(NormParams p) {
    const int D = (int)p.D;
    constexpr int N = EL / V;
    __shared__ float part[2][kMaxWarps];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    const E *x = static_cast<const E *>(p.x) + row * p.xs;
    float f[N][V];
    {
        Pack<E, V> raw[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (live && column<V>(k) < D) raw[k] = ld_pack<E, V>(x + column<V>(k));
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (live && column<V>(k) < D) unpack<E, V>(raw[k], f[k]);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) f[k][v] = 0.f;
        }
    }
    const float inv = 1.f / (float)p.D;
    const float mean = row_sum(lane_sum(reinterpret_cast<const float (&)[EL]>(f)), part[0]) * inv;
    float sq[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sq[v] = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (column<V>(k) >= D) continue;
        fma_n<V>(f[k], f[k], 1.f, -mean);
        fma_n<V>(sq, f[k], f[k], sq);
    }
    const float var = row_sum(lane_sum(sq), part[1]) * inv;
    if (!live) return;
    const float rstd = 1.f / sqrtf(var + p.eps);
    E *out = static_cast<E *>(p.out) + row * p.os;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int c = column<V>(k);
        if (c >= D) continue;
        float w[V], b[V];
        ld_param<V>(p.weight, c, 1.f, w);
        ld_param<V>(p.bias, c, 0.f, b);
        fma_n<V>(f[k], f[k], rstd, 0.f);
        fma_n<V>(f[k], f[k], w, b);
        st_f<E, V>(out + c, f[k]);
    }
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
}

constexpr int kStages = 3;   // rows of a copy ring

// Many rows: persistent CTAs, the next two rows on their way into the threads' own slots of
// shared memory, the weights in registers.  8192 x 8192 bf16: 49 us, 5.5 TB/s (a plain copy
// of the same bytes 47 us).
template <typename E, int V, int EL>
__global__ void __launch_bounds__(256, 2) norm_fwd_stream_kernel(NormParams p) {
    const int D = (int)p.D;
    constexpr int N = EL / V;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float part[4][kMaxWarps];
    const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
    Pack<E, V> *ring = reinterpret_cast<Pack<E, V> *>(smem);   // [stage][group][thread]
    const auto slot = [&](int stage, int k) -> Pack<E, V> & { return ring[(stage * N + k) * threads + tid]; };
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const auto fetch = [&](int64_t row, int stage) {
        if (row < p.rows) {
            const E *x = static_cast<const E *>(p.x) + row * p.xs;
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (column<V>(k) < D) copy_async<sizeof(E) * V>(&slot(stage, k), x + column<V>(k));
        }
        copies_commit();
    };
    float w[N][V], b[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v) w[k][v] = b[k][v] = 0.f;
        if (column<V>(k) >= D) {   // columns that do not exist stay 0 in every slot
            for (int stage = 0; stage < kStages; ++stage) st_f<E, V>(&slot(stage, k).e[0], w[k]);
            continue;
        }
        ld_param<V>(p.weight, column<V>(k), 1.f, w[k]);
        ld_param<V>(p.bias, column<V>(k), 0.f, b[k]);
    }
    const float inv = 1.f / (float)D;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int passes = (int)ceil_div(p.rows - (int64_t)blockIdx.x * blockDim.y, step);
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(row + k * step, k);
    for (int pass = 0, stage = 0; pass < passes; ++pass, row += step) {
        fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        copies_wait<kStages - 1>();   // this thread's own copies: no barrier needed
        float f[N][V];
#pragma unroll
        for (int k = 0; k < N; ++k) unpack<E, V>(slot(stage, k), f[k]);
        const float mean = row_sum(lane_sum(reinterpret_cast<const float (&)[EL]>(f)), part[2 * (pass & 1)]) * inv;
        float sq[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sq[v] = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (column<V>(k) >= D) continue;
            fma_n<V>(f[k], f[k], 1.f, -mean);
            fma_n<V>(sq, f[k], f[k], sq);
        }
        const float rstd = 1.f / sqrtf(fmaf(row_sum(lane_sum(sq), part[2 * (pass & 1) + 1]), inv, p.eps));
        stage = stage + 1 == kStages ? 0 : stage + 1;
        if (row >= p.rows) continue;
        E *out = static_cast<E *>(p.out) + row * p.os;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (column<V>(k) >= D) continue;
            fma_n<V>(f[k], f[k], rstd, 0.f);
            fma_n<V>(f[k], f[k], w[k], b[k]);
            st_f<E, V>(out + column<V>(k), f[k]);
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
    }
    copies_wait<0>();
}

// One CTA of 512 threads per SM, rows of x and dout two ahead in the ring.  8192 x 8192 bf16:
// 85 us with the sums over CTAs (6 us), 4.7 TB/s; bound by issue and the reductions.  With
// 1024 threads of half the elements the registers spill: 141 us; with one row finished while
// the next one's sums form: 87 us.
template <typename E, int V, int EL>
__global__ void __launch_bounds__(512, 1) norm_bwd_kernel(NormParams p, float *part_out) {
    const int D = (int)p.D;
    constexpr int N = EL / V;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float part[2][2][kMaxWarps];
    __shared__ float2 stats[kStages][kMaxWarps];
    const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x, warp = tid >> 5;
    Pack<E, V> *ring = reinterpret_cast<Pack<E, V> *>(smem);   // [stage][x, dy][group][thread]
    const auto slot = [&](int stage, int t, int k) -> Pack<E, V> & { return ring[((stage * 2 + t) * N + k) * threads + tid]; };
    const int64_t step = (int64_t)gridDim.x * blockDim.y;

    auto fetch = [&](int64_t row, int stage) {
        if (row < p.rows) {
            const E *x = static_cast<const E *>(p.x) + row * p.xs, *dy = static_cast<const E *>(p.dout) + row * p.ds;
            if constexpr (sizeof(E) * V == 2) {
                E t[2 * N];
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (column<V>(k) < D) t[2 * k] = x[column<V>(k)], t[2 * k + 1] = dy[column<V>(k)];
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (column<V>(k) < D) slot(stage, 0, k).e[0] = t[2 * k], slot(stage, 1, k).e[0] = t[2 * k + 1];
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    if (column<V>(k) < D) {
                        copy_async<sizeof(E) * V>(&slot(stage, 0, k), x + column<V>(k));
                        copy_async<sizeof(E) * V>(&slot(stage, 1, k), dy + column<V>(k));
                    }
                }
            }
            if ((tid & 31) == 0) {
                copy_async<4>(&stats[stage][warp].x, p.mean + row);
                copy_async<4>(&stats[stage][warp].y, p.rstd + row);
            }
        }
        copies_commit();
    };

    // columns that do not exist stay 0 in every slot
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (column<V>(k) < D) continue;
        for (int j = 0; j < 2 * kStages; ++j) {
            const float zero[V] = {};
            st_f<E, V>(&slot(j / 2, j % 2, k).e[0], zero);
        }
    }
    float w[EL], dw[EL], db[EL];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float t[V] = {};
        if (column<V>(k) < D) ld_param<V>(p.weight, column<V>(k), 1.f, t);
#pragma unroll
        for (int v = 0; v < V; ++v) w[k * V + v] = t[v], dw[k * V + v] = db[k * V + v] = 0.f;
    }
    const float inv = 1.f / (float)p.D;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int passes = (int)ceil_div(p.rows - (int64_t)blockIdx.x * blockDim.y, step);
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(row + k * step, k);
    for (int pass = 0, stage = 0; pass < passes; ++pass, row += step) {
        fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        copies_wait<kStages - 1>();
        __syncwarp();
        const bool live = row < p.rows;
        const float2 st = stats[stage][warp];
        float xh[EL], d[EL], s1 = 0.f, s2 = 0.f;
        if (live) {
            float t[EL];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                unpack<E, V>(slot(stage, 0, k), reinterpret_cast<float (&)[V]>(xh[k * V]));
                unpack<E, V>(slot(stage, 1, k), reinterpret_cast<float (&)[V]>(d[k * V]));
            }
            fma_n<EL>(xh, xh, 1.f, -st.x);
            fma_n<EL>(xh, xh, st.y, 0.f);
            fma_n<EL>(dw, d, xh, dw);
            add_n<EL>(db, db, d);
            mul_n<EL>(d, d, w);
            mul_n<EL>(t, d, xh);
            s1 = lane_sum(d);
            s2 = lane_sum(t);
        }
        row_sum2(s1, s2, part[pass & 1]);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        if (!live) continue;
        // rstd (d - m1 - xh m2)
        fma_n<EL>(xh, xh, -st.y * s2 * inv, -st.y * s1 * inv);
        const float r = st.y;
#pragma unroll
        for (int e = 0; e < EL; e += 2) {
            const float2 o = sm103::fma2(make_float2(d[e], d[e + 1]), both(r), make_float2(xh[e], xh[e + 1]));
            d[e] = o.x, d[e + 1] = o.y;
        }
        E *dx = static_cast<E *>(p.dx) + row * p.D;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (column<V>(k) < D) st_f<E, V>(dx + column<V>(k), reinterpret_cast<const float (&)[V]>(d[k * V]));
    }
    copies_wait<0>();
    if (!part_out) return;
    // over the CTA's rows side by side, one after the other
    float *sums = reinterpret_cast<float *>(smem);   // [2][EL][blockDim.x], over the ring
    for (int y = 0; y < (int)blockDim.y; ++y) {
        __syncthreads();
        if ((int)threadIdx.y != y) continue;
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            float *at = sums + e * blockDim.x + threadIdx.x;
            if (y > 0) dw[e] += at[0], db[e] += at[EL * blockDim.x];
            if (y + 1 < (int)blockDim.y) at[0] = dw[e], at[EL * blockDim.x] = db[e];
        }
    }
    if (threadIdx.y == blockDim.y - 1) {
        float *at = part_out + (int64_t)blockIdx.x * 2 * p.D;
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            const int c = column<V>(e / V) + e % V;
            if (c < D) at[c] = dw[e], at[p.D + c] = db[e];
        }
    }
}

// ---- rows too long for a thread's registers: a CTA per row, several passes (the later ones
// through L2), V elements at a time
constexpr int kLongThreads = 512;

template <typename E, int V>
__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(NormParams p) {
    __shared__ float part[2][kMaxWarps];
    const int D = (int)p.D, c0 = threadIdx.x * V;
    constexpr int kStep = kLongThreads * V;
    const int64_t row = blockIdx.x;
    const E *x = static_cast<const E *>(p.x) + row * p.xs;
    E *out = static_cast<E *>(p.out) + row * p.os;
    const float inv = 1.f / (float)D;
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 0.f;
#pragma unroll 4
    for (int64_t c = c0; c < D; c += kStep) {
        float f[V];
        ld_f<E, V>(x + c, f);
        add_n<V>(s, s, f);
    }
    const float mean = row_sum(lane_sum(s), part[0]) * inv;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 0.f;
#pragma unroll 4
    for (int64_t c = c0; c < D; c += kStep) {
        float f[V];
        ld_f<E, V>(x + c, f);
        fma_n<V>(f, f, 1.f, -mean);
        fma_n<V>(s, f, f, s);
    }
    const float rstd = 1.f / sqrtf(fmaf(row_sum(lane_sum(s), part[1]), inv, p.eps));
#pragma unroll 2
    for (int64_t c = c0; c < D; c += kStep) {
        float f[V], w[V], b[V];
        ld_f<E, V>(x + c, f);
        ld_param<V>(p.weight, (int)c, 1.f, w);
        ld_param<V>(p.bias, (int)c, 0.f, b);
        fma_n<V>(f, f, 1.f, -mean);
        fma_n<V>(f, f, rstd, 0.f);
        fma_n<V>(f, f, w, b);
        st_f<E, V>(out + c, f);
    }
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
}

template <typename E, int V>
__global__ void __launch_bounds__(kLongThreads) norm_bwd_long_kernel(NormParams p) {
    __shared__ float part[2][kMaxWarps];
    const int D = (int)p.D, c0 = threadIdx.x * V;
    constexpr int kStep = kLongThreads * V;
    const int64_t row = blockIdx.x;
    const E *x = static_cast<const E *>(p.x) + row * p.xs, *dy = static_cast<const E *>(p.dout) + row * p.ds;
    E *dx = static_cast<E *>(p.dx) + row * p.D;
    const float mean = p.mean[row], rstd = p.rstd[row], inv = 1.f / (float)D;
    float s1[V], s2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s1[v] = s2[v] = 0.f;
#pragma unroll 2
    for (int64_t c = c0; c < D; c += kStep) {
        float f[V], d[V], w[V];
        ld_f<E, V>(x + c, f);
        ld_f<E, V>(dy + c, d);
        ld_param<V>(p.weight, (int)c, 1.f, w);
        fma_n<V>(f, f, 1.f, -mean);
        fma_n<V>(f, f, rstd, 0.f);
        mul_n<V>(d, d, w);
        add_n<V>(s1, s1, d);
        fma_n<V>(s2, d, f, s2);
    }
    const float m1 = row_sum(lane_sum(s1), part[0]) * inv, m2 = row_sum(lane_sum(s2), part[1]) * inv;
#pragma unroll 2
    for (int64_t c = c0; c < D; c += kStep) {
        float f[V], d[V], w[V];
        ld_f<E, V>(x + c, f);
        ld_f<E, V>(dy + c, d);
        ld_param<V>(p.weight, (int)c, 1.f, w);
        fma_n<V>(f, f, 1.f, -mean);
        fma_n<V>(f, f, rstd, 0.f);
        mul_n<V>(d, d, w);
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = rstd * (d[v] - fmaf(f[v], m2, m1));
        st_f<E, V>(dx + c, d);
    }
}

// A thread per V columns, blockIdx.y a block of rows.
template <typename E, int V>
__global__ void __launch_bounds__(128) norm_param_part_kernel(NormParams p, int64_t block_rows, float *part_out) {
    const int64_t c = ((int64_t)blockIdx.x * 128 + threadIdx.x) * V, r0 = blockIdx.y * block_rows, r1 = min(r0 + block_rows, p.rows);
    if (c >= p.D) return;
    float w[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = b[v] = 0.f;
    const E *x = static_cast<const E *>(p.x) + c, *dy = static_cast<const E *>(p.dout) + c;
#pragma unroll 4
    for (int64_t row = r0; row < r1; ++row) {
        float f[V], d[V];
        ld_f<E, V>(x + row * p.xs, f);
        ld_f<E, V>(dy + row * p.ds, d);
        fma_n<V>(f, f, 1.f, -p.mean[row]);
        fma_n<V>(f, f, p.rstd[row], 0.f);
        fma_n<V>(w, d, f, w);
        add_n<V>(b, b, d);
    }
    float *at = part_out + blockIdx.y * 2 * p.D + c;
#pragma unroll
    for (int v = 0; v < V; ++v) at[v] = w[v], at[p.D + v] = b[v];
}

// part [parts, 2, D] to dweight, dbias.
__global__ void __launch_bounds__(kSumThreads) norm_param_sum_kernel(NormParams p, int64_t parts, const float *part) {
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const float t = column_sum(part, parts, 2 * p.D, c, c < 2 * p.D);
    if (threadIdx.x >= 32) return;
    if (c < p.D) {
        if (p.dweight) p.dweight[c] = t;
    } else if (c < 2 * p.D) {
        if (p.dbias) p.dbias[c - p.D] = t;
    }
}

// ---- host side
constexpr int64_t kFwdMaxD = 16384, kBwdMaxD = 8192;
constexpr int64_t kLongParts = 256;

// Threads of a row, and rows of a CTA: at most `most` threads, whole warps.
dim3 row_block(int64_t D, int el, int most) {
    const int x = (int)(ceil_div(D, 32 * el) * 32);
    return dim3(x, x >= most ? 1 : most / x);
}

// 16-byte groups where every row allows them.
bool aligned_rows(const NormParams &p, const void *a, int64_t as, const void *b, int64_t bs) {
    const int64_t V = 16 / (int64_t)dtype_bytes(p.dtype);
    const void *ptrs[] = {p.x, a, b, p.weight, p.bias};
    for (const void *q : ptrs)
        if (reinterpret_cast<uintptr_t>(q) % 16) return false;
    return p.D % V == 0 && p.xs % V == 0 && as % V == 0 && bs % V == 0;
}

bool wants_params(const NormParams &p) { return p.dweight || p.dbias; }

// Backward: 16 elements per thread; 8 for rows that then still fit a CTA.
int bwd_el(const NormParams &p) { return p.D <= 512 * 8 ? 8 : 16; }
int64_t bwd_grid(const NormParams &p, int sms) {
    return std::min(ceil_div(p.rows, (int64_t)row_block(p.D, bwd_el(p), 512).y), (int64_t)sms);
}
// Rows of more than 8192 elements, and of more than 4096 in 16 bits that are not aligned:
// their 2-byte elements pass through registers on the way to the ring, and with 16 of them
// per thread that spills.  8192 rows of 8191 bf16: 595 us, in several passes 313 us; of
// 4097: 524 and 177; but of 1537, at 8 per thread: 52 and 75.
bool long_rows(const NormParams &p) {
    return p.D > kBwdMaxD || (p.D > 4096 && p.dtype != kFP32 && !aligned_rows(p, p.dout, p.ds, p.dx, 0));
}
int64_t bwd_parts(const NormParams &p, int sms) {
    if (p.rows == 0) return 0;
    return !long_rows(p) ? bwd_grid(p, sms) : std::min(ceil_div(p.rows, 64), kLongParts);
}

template <typename E, int V, int EL>
cudaError_t run_fwd(const NormParams &p, cudaStream_t stream) {
    const dim3 block = row_block(p.D, EL, 256);
    norm_fwd_kernel<E, V, EL><<<(unsigned)ceil_div(p.rows, (int64_t)block.y), block, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename E, int V, int EL>
cudaError_t run_fwd_stream(const NormParams &p, int sms, cudaStream_t stream) {
    const dim3 block = row_block(p.D, EL, 256);
    constexpr auto kernel = norm_fwd_stream_kernel<E, V, EL>;
    const cudaError_t e = allow_smem<kernel>(256 * EL * kStages * (int)sizeof(E));
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min(ceil_div(p.rows, (int64_t)block.y), (int64_t)sms * 2);
    kernel<<<(unsigned)grid, block, block.x * block.y * EL * kStages * (int)sizeof(E), stream>>>(p);
    return cudaGetLastError();
}

template <typename E, int V, int EL>
cudaError_t run_bwd(const NormParams &p, float *part, int sms, cudaStream_t stream) {
    const dim3 block = row_block(p.D, EL, 512);
    const int threads = block.x * block.y;
    const int smem = threads * EL * std::max(kStages * 2 * (int)sizeof(E), block.y > 1 ? 8 : 0);
    constexpr auto kernel = norm_bwd_kernel<E, V, EL>;
    const cudaError_t e = allow_smem<kernel>(512 * EL * kStages * 2 * (int)sizeof(E));
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)bwd_grid(p, sms), block, smem, stream>>>(p, part);
    return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_scratch_bytes(const NormParams &p, int sms) {
    return wants_params(p) ? (size_t)(bwd_parts(p, sms) * 2 * p.D) * sizeof(float) : 0;
}

cudaError_t launch_norm_fwd(const NormParams &p, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        constexpr int V = 16 / sizeof(E);
        if (p.D > kFwdMaxD) {
            if (aligned_rows(p, p.out, p.os, nullptr, 0)) norm_fwd_long_kernel<E, V><<<(unsigned)p.rows, kLongThreads, 0, stream>>>(p);
            else norm_fwd_long_kernel<E, 1><<<(unsigned)p.rows, kLongThreads, 0, stream>>>(p);
            return cudaGetLastError();
        }
        // elements per thread: a warp to a short row; of longer ones many, or few where few
        // rows leave most of the GPU idle
        const int el = p.D <= 256 ? 8 : p.D <= 512 ? 16 : p.rows <= 4 * sms && p.D <= 8192 ? 8 : 32;
        const bool aligned = aligned_rows(p, p.out, p.os, nullptr, 0);
        // many rows: the streaming kernel.  8192 x 8192 bf16: 50 us against 62 us; in 32 bits
        // its ring and registers leave too few bytes on their way: 96 us against 84 us
        if constexpr (sizeof(E) == 2) {
            if (aligned && p.D > 512 && p.D <= 256 * 32 && p.rows >= 8 * sms * (int64_t)row_block(p.D, 32, 256).y)
                return run_fwd_stream<E, V, 32>(p, sms, stream);
        }
        if (aligned) return el == 8 ? run_fwd<E, V, 8>(p, stream) : el == 16 ? run_fwd<E, V, 16>(p, stream) : run_fwd<E, V, 32>(p, stream);
        // single elements: at most 16 to a thread.  8192 x 8191 bf16: 134 us, 167 with 32, 199
        // with 8; 8192 x 1537: 31, 42 with 32
        return el == 8 ? run_fwd<E, 1, 8>(p, stream) : run_fwd<E, 1, 16>(p, stream);
    });
}

cudaError_t launch_norm_bwd(const NormParams &p, unsigned char *ws, int sms, cudaStream_t stream) {
    const int64_t parts = bwd_parts(p, sms);
    float *part = wants_params(p) ? reinterpret_cast<float *>(ws) : nullptr;
    const cudaError_t e = with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        constexpr int V = 16 / sizeof(E);
        if (p.rows == 0) return cudaSuccess;
        const bool wide = aligned_rows(p, p.dout, p.ds, p.dx, 0);
        if (long_rows(p)) {
            const auto run_long = [&](auto v) {
                constexpr int LV = decltype(v)::value;
                norm_bwd_long_kernel<E, LV><<<(unsigned)p.rows, kLongThreads, 0, stream>>>(p);
                if (part)
                    norm_param_part_kernel<E, LV><<<dim3((unsigned)ceil_div(p.D, 128 * LV), (unsigned)parts), 128, 0, stream>>>(
                        p, ceil_div(p.rows, parts), part);
                return cudaGetLastError();
            };
            return wide ? run_long(std::integral_constant<int, V>{}) : run_long(std::integral_constant<int, 1>{});
        }
        if (bwd_el(p) == 8) return wide ? run_bwd<E, V, 8>(p, part, sms, stream) : run_bwd<E, 1, 8>(p, part, sms, stream);
        if constexpr (sizeof(E) == 4)
            if (!wide) return run_bwd<E, 1, 16>(p, part, sms, stream);
        return run_bwd<E, V, 16>(p, part, sms, stream);
    });
    if (e != cudaSuccess) return e;
    if (part || (wants_params(p) && p.rows == 0))
        norm_param_sum_kernel<<<(unsigned)ceil_div(2 * p.D, 32), kSumThreads, 0, stream>>>(p, parts, part);
    return cudaGetLastError();
}

}  // namespace kda
