// RMS norm over the last axis, forward and backward.
//   h = x + residual, rounded to the tensors' type;  y = h rstd w,  rstd = 1 / sqrt(mean(h^2) + eps)
//   with d = dy w, hat = h rstd:  dx = rstd (d - hat mean(d hat)) + dresidual,
//   dw = sum over rows of dy hat
// Sums are fp32.  h is rounded before it is normed, so that what the residual stream keeps is
// what the output belongs to, and the backward pass starts from it.  8-bit outputs have a scale
// for each block of 128 columns (fp8_io.cuh).
//
// Both directions move each value once.  Forward, the threads blockDim.x share a row (blockDim.y
// rows per CTA), each with 8 to 32 of its elements in registers from the load to the store.
// Backward, CTAs are persistent: a thread's columns stay the same, so that its weights and their
// gradients stay in registers, and the next rows are on their way into shared memory.  Rows that
// are not aligned, or too long for registers, take kernels of their own.
//
// 8192 x 8192 bf16 with a residual: forward 79 us to 8 bits (5.9 TB/s) and 80.9 us to bf16 (6.6, a
// plain copy's rate), bound by memory; backward 82 us (6.5 TB/s; 76 us without the weight's gradient):
// issue 53% at 16 warps per SM.  With 16 elements per thread the backward pass took 121 us, as each
// row costs a thread some 150 instructions beside those of its elements.  8192 x 8192 fp32 158 us forward
// and 156 backward (6.8 and 6.9 TB/s).  4999 x 1537 fp16, unaligned, forward 10.8 us (2.9 TB/s), with a
// residual backward 27.7 us (2.2): element-wise loads and stores.  Rows too long for registers backward
// pass over x and dout three times: 4096 x 16384 fp32 328 us (3.3 TB/s).
#include <algorithm>
#include <initializer_list>
#include <utility>

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

// ---- rows in registers: N groups of V = 16 bytes to a thread, neighbouring threads side by side

// Sum over the blockDim.x threads of every row of the CTA; all threads of the CTA call it together.
__device__ __forceinline__ float row_sum(float v, float (&part)[32]) {
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
template <int V>
__device__ __forceinline__ int column(int k) { return (k * blockDim.x + threadIdx.x) * V; }

// A group of 8-bit outputs: V values that with those of the 128 / V threads around make a block.
template <bool E5M2, int V>
__device__ __forceinline__ void st_group_fp8(uint8_t *at, uint8_t *scale, float (&f)[V], bool in) {
    bool special = false;
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, finite_abs(f[j], special));
#pragma unroll
    for (int o = 64 / V; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!in) return;
    const int e = scale_byte(top, E5M2);
    if (threadIdx.x % (128 / V) == 0) *scale = (uint8_t)e;
    scale_n(f, inverse_scale(e));
    Pack<uint32_t, V / 4> w;
#pragma unroll
    for (int j = 0; j < V; j += 4) w.e[j / 4] = quad_to_fp8<E5M2>(f[j], f[j + 1], f[j + 2], f[j + 3], special);
    *reinterpret_cast<Pack<uint32_t, V / 4> *>(at) = w;
}

// OUT: 0 = out in E, 4, 5 = in 8 bits (kE4M3, kE5M2).
template <typename E, int EL, int OUT>
__global__ void __launch_bounds__(512) rms_fwd_row_kernel(RmsParams p) {
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    constexpr int V = 16 / sizeof(E), N = EL / V;
    __shared__ float part[32];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int D = row < p.rows ? (int)p.D : 0;            // rows behind the last take part in the barriers only
    const E *x = static_cast<const E *>(p.x) + row * p.xs;
    Pack<E, V> h[N], r[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (column<V>(k) < D) h[k] = ld_pack<E, V>(x + column<V>(k));
    if (p.res) {
        const E *res = static_cast<const E *>(p.res) + row * p.rs;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (column<V>(k) < D) r[k] = ld_pack<E, V>(res + column<V>(k));
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float a[V], b[V];
            unpack<E, V>(h[k], a);
            unpack<E, V>(r[k], b);
            add_n<V>(a, a, b);
            st_f<E, V>(h[k].e, a);
        }
        if (p.res_out) {
            E *sum = static_cast<E *>(p.res_out) + row * p.ros;
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (column<V>(k) < D) *reinterpret_cast<Pack<E, V> *>(sum + column<V>(k)) = h[k];
        }
    }
    // Few rows: the weights are asked for before the row's sum is waited for (64 x 2048 bf16 1.85 us
    // instead of 2.05; with more in registers it does not pay, nor in fp32).
    constexpr bool kEarly = EL == 8 && sizeof(E) == 2;
    float w[kEarly ? EL : V];
    const auto weights = [&](int k, float (&to)[V]) {
#pragma unroll
        for (int j = 0; j < V; j += 4) ld_f<float, 4>(p.weight + column<V>(k) + j, reinterpret_cast<float (&)[4]>(to[j]));
    };
    if constexpr (kEarly) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (p.weight && column<V>(k) < D) weights(k, reinterpret_cast<float (&)[V]>(w[k * V]));
    }
    float s[V], t = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (column<V>(k) >= D) continue;
        float a[V];
        unpack<E, V>(h[k], a);
        fma_n<V>(s, a, a, s);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) t += s[j];
    const float rstd = 1.f / sqrtf(row_sum(t, part) / (float)(int)p.D + p.eps);
    if (threadIdx.x == 0 && D && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int c = column<V>(k);
        const bool in = c < D;
        if (OUT == 0 && !in) continue;
        float a[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = 0.f;
        if (in) {
            unpack<E, V>(h[k], a);
            scale_n(a, rstd);
            if (p.weight) {
                float (&f)[V] = reinterpret_cast<float (&)[V]>(w[kEarly ? k * V : 0]);
                if constexpr (!kEarly) weights(k, f);
                mul_n<V>(a, a, f);
            }
        }
        if constexpr (OUT == 0) st_f<E, V>(static_cast<E *>(p.out) + row * p.os + c, a);
        else st_group_fp8<OUT == kE5M2, V>(static_cast<uint8_t *>(p.out) + row * p.os + c, p.scales + row * p.ss + c / kFp8Block, a, in);
    }
}

// ---- backward, persistent: blockDim.y rows at once, each with a ring and a barrier of its own, so
// that one row's sums form while another is stored

constexpr int kBwdThreads = 512;
constexpr int kFewCtas = 8;   // of a cluster that has all rows
// Most elements per thread, and rows in its ring (up to 4, in 192 KB).
template <typename E> constexpr int kBwdMost = sizeof(E) == 4 ? 16 : 32;
template <typename E, int EL> constexpr int kBwdStages = std::min(4, 192 * 1024 / (kBwdThreads * EL * 3 * (int)sizeof(E)));

// Sum over the CTA's rows side by side, in their order, to its part; a thread takes whole columns.
// (One row after the other, with a barrier between them, took 6 us of 18 at 4096 x 1024.)  A cluster
// joins its CTAs' sums through distributed shared memory, and has the gradient.
__device__ __forceinline__ void sum_side_by_side(float *sums, int stride, int D, float *part_out) {
    const int threads = blockDim.x * blockDim.y, ctas = (int)sm103::cluster_size();
    float *out = ctas > 1 ? sums : part_out + (int64_t)blockIdx.x * D;
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < D; c += threads) {
        float t = 0.f;
#pragma unroll 4
        for (int y = 0; y < (int)blockDim.y; ++y) t += sums[y * stride + c];
        out[c] = t;
    }
    if (ctas == 1) return;
    __syncwarp();
    sm103::cluster_sync();
    const uint32_t at = sm103::smem_u32(sums);
    for (int c = (int)sm103::cluster_ctarank() * threads + threadIdx.y * blockDim.x + threadIdx.x; c < D; c += ctas * threads) {
        float v[kFewCtas], t = 0.f;
#pragma unroll
        for (int q = 0; q < kFewCtas; ++q) v[q] = q < ctas ? sm103::ld_cluster(sm103::mapa_shared(at + 4 * c, q)) : 0.f;
#pragma unroll
        for (int q = 0; q < kFewCtas; ++q) t += v[q];
        part_out[c] = t;
    }
    __syncwarp();
    sm103::cluster_sync();   // the others have read
}

template <typename E, int EL>
__global__ void __launch_bounds__(kBwdThreads, 1) rms_bwd_row_kernel(RmsParams p, float *part_out) {
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    constexpr int V = 16 / sizeof(E), N = EL / V, kStages = kBwdStages<E, EL>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float part[2][32];
    const int D = (int)p.D, threads = blockDim.x * blockDim.y, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool more = p.dres != nullptr;
    const float inv = 1.f / (float)D;
    // group k of tensor t of stage s is ring[((3 s + t) N + k) threads]
    Pack<E, V> *ring = reinterpret_cast<Pack<E, V> *>(smem) + threadIdx.y * blockDim.x + threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t ahead = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;      // the next row to ask for
    const auto request = [&](int stage) {
        if (ahead < p.rows) {
            const E *h = static_cast<const E *>(p.x) + ahead * p.xs, *g = static_cast<const E *>(p.dout) + ahead * p.ds;
            const E *r = static_cast<const E *>(p.dres) + ahead * p.drs;
            Pack<E, V> *to = ring + stage * 3 * N * threads;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int c = column<V>(k);
                if (c >= D) continue;
                copy_async<16>(to + k * threads, h + c);
                copy_async<16>(to + (N + k) * threads, g + c);
                if (more) copy_async<16>(to + (2 * N + k) * threads, r + c);
            }
        }
        ahead += step;
        copies_commit();
    };
    float w[EL], dw[EL];
#pragma unroll
    for (int k = 0; k < EL; k += 4) {
        const int c = column<V>(k / V) + k % V;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[k + j] = 1.f, dw[k + j] = 0.f;
        if (p.weight && c < D) ld_f<float, 4>(p.weight + c, reinterpret_cast<float (&)[4]>(w[k]));
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) request(i);
    int stage = 0, turn = 0;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    float next = row < p.rows ? p.rstd[row] : 0.f;
    for (; row < p.rows; row += step) {
        request(stage == 0 ? kStages - 1 : stage - 1);
        const float rstd = next;
        if (row + step < p.rows) next = p.rstd[row + step];
        copies_wait<kStages - 1>();
        const Pack<E, V> *at = ring + stage * 3 * N * threads;
        float s[V], t = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (column<V>(k) >= D) continue;
            float h[V], g[V];
            float (&ww)[V] = reinterpret_cast<float (&)[V]>(w[k * V]), (&dd)[V] = reinterpret_cast<float (&)[V]>(dw[k * V]);
            unpack<E, V>(at[k * threads], h);
            unpack<E, V>(at[(N + k) * threads], g);
            scale_n(h, rstd);
            fma_n<V>(dd, g, h, dd);
            mul_n<V>(g, g, ww);
            fma_n<V>(s, g, h, s);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) t += s[j];
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (warps > 1) {
            float *sums = part[turn] + threadIdx.y * warps;
            if (lane == 0) sums[threadIdx.x >> 5] = t;
            sm103::named_bar(1 + threadIdx.y, blockDim.x);
            t = lane < warps ? sums[lane] : 0.f;
#pragma unroll
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            turn ^= 1;
        }
        // dx = rstd d - (rstd^2 mean) h + dresidual
        const float mean = t * inv, c2 = -rstd * rstd * mean;
        E *dx = static_cast<E *>(p.dx) + row * p.D;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (column<V>(k) >= D) continue;
            float h[V], g[V];
            unpack<E, V>(at[k * threads], h);
            unpack<E, V>(at[(N + k) * threads], g);
            scale_n(h, c2);
            if (more) {
                float f[V];
                unpack<E, V>(at[(2 * N + k) * threads], f);
                add_n<V>(h, h, f);
            }
            mul_n<V>(g, g, reinterpret_cast<float (&)[V]>(w[k * V]));
            const float2 r = both(rstd);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float2 o = sm103::fma2(make_float2(g[j], g[j + 1]), r, make_float2(h[j], h[j + 1]));
                g[j] = o.x, g[j + 1] = o.y;
            }
            st_f<E, V>(dx + column<V>(k), g);
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();
    if (!part_out) return;
    // Rows side by side: each leaves its gradients over the ring, as groups of 4 columns.
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem);   // [blockDim.y][EL blockDim.x]
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float *d = dw + k * V + j;
            if (column<V>(k) < D)
                *reinterpret_cast<float4 *>(sums + threadIdx.y * EL * blockDim.x + column<V>(k) + j) = make_float4(d[0], d[1], d[2], d[3]);
        }
    __syncthreads();
    sum_side_by_side(sums, EL * blockDim.x, D, part_out);
}

// ---- rows that are not aligned: a warp takes blocks of 128 columns, 4 columns 32 apart to a lane, NB
// blocks that it keeps in registers; blockDim.x threads to a row, blockDim.y rows per CTA

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


template <typename E, int NB, int OUT>
__global__ void __launch_bounds__(512) rms_fwd_odd_kernel(RmsParams p) {
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    __shared__ float part[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t D = row < p.rows ? p.D : 0;
    const E *x = static_cast<const E *>(p.x) + row * p.xs, *res = static_cast<const E *>(p.res) + row * p.rs;
    E *sum = static_cast<E *>(p.res_out) + row * p.ros;
    float h[NB][4], s = 0.f;
#pragma unroll
    for (int k = 0; k < NB; ++k) ld_block<E, false>(x, (int64_t)(warp + k * warps) * kFp8Block, D, lane, h[k]);
    if (p.res) {
        float f[NB][4];   // all of them before the first store, which may be over them
#pragma unroll
        for (int k = 0; k < NB; ++k) ld_block<E, false>(res, (int64_t)(warp + k * warps) * kFp8Block, D, lane, f[k]);
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) h[k][j] = to_f(from_f<E>(h[k][j] + f[k][j]));
        if (p.res_out) {
#pragma unroll
            for (int k = 0; k < NB; ++k) st_block<E, false>(sum, (int64_t)(warp + k * warps) * kFp8Block, D, lane, h[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(h[k][j], h[k][j], s);
    const float rstd = 1.f / sqrtf(row_sum(s, part) / (float)(int)p.D + p.eps);
    if (D == 0) return;
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        const int64_t b = warp + k * warps, c0 = b * kFp8Block;
        if (c0 >= D) break;
        float w[4];
        if (p.weight) ld_block<float, false>(p.weight, c0, D, lane, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] *= p.weight ? rstd * w[j] : rstd;
        if constexpr (OUT == 0) st_block<E, false>(static_cast<E *>(p.out) + row * p.os, c0, D, lane, h[k]);
        else st_block_fp8<OUT == kE5M2, false>(static_cast<uint8_t *>(p.out) + row * p.os, p.scales + row * p.ss + b, c0, D, lane, h[k], false);
    }
}

// Persistent, like the aligned rows' kernel, with the weights and their gradients in registers; the
// next row's loads are left to the other CTAs of the SM.
template <typename E, int NB>
__global__ void __launch_bounds__(512) rms_bwd_odd_kernel(RmsParams p, float *part_out) {
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    __shared__ float part[2][32];
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const float inv = 1.f / (float)(int)p.D;
    float w[NB][4], dw[NB][4];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[k][j] = 1.f, dw[k][j] = 0.f;
        if (p.weight) ld_block<float, false>(p.weight, (int64_t)(warp + k * warps) * kFp8Block, p.D, lane, w[k]);
    }
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * blockDim.y; first < p.rows; first += (int64_t)gridDim.x * blockDim.y) {
        const int64_t row = first + threadIdx.y, D = row < p.rows ? p.D : 0;
        const E *x = static_cast<const E *>(p.x) + row * p.xs, *dy = static_cast<const E *>(p.dout) + row * p.ds;
        const E *dres = static_cast<const E *>(p.dres) + row * p.drs;
        float h[NB][4], g[NB][4], s = 0.f;
#pragma unroll
        for (int k = 0; k < NB; ++k) ld_block<E, false>(x, (int64_t)(warp + k * warps) * kFp8Block, D, lane, h[k]);
#pragma unroll
        for (int k = 0; k < NB; ++k) ld_block<E, false>(dy, (int64_t)(warp + k * warps) * kFp8Block, D, lane, g[k]);
        const float rstd = D ? p.rstd[row] : 0.f;
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[k][j] *= rstd;
                dw[k][j] = fmaf(g[k][j], h[k][j], dw[k][j]);
                g[k][j] *= w[k][j];
                s = fmaf(g[k][j], h[k][j], s);
            }
        float f[NB][4];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[k][j] = 0.f;
            if (p.dres) ld_block<E, false>(dres, (int64_t)(warp + k * warps) * kFp8Block, D, lane, f[k]);
        }
        const float mean = row_sum(s, part[turn]) * inv;
        turn ^= 1;
        E *dx = static_cast<E *>(p.dx) + row * p.D;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[k][j] = fmaf(rstd, fmaf(-mean, h[k][j], g[k][j]), f[k][j]);
            st_block<E, false>(dx, (int64_t)(warp + k * warps) * kFp8Block, D, lane, f[k]);
        }
    }
    if (!part_out) return;
    float *sums = reinterpret_cast<float *>(smem) + threadIdx.y * 4 * NB * blockDim.x;   // [blockDim.y][4 NB blockDim.x]
#pragma unroll
    for (int k = 0; k < NB; ++k) st_block<float, false>(sums, (int64_t)(warp + k * warps) * kFp8Block, p.D, lane, dw[k]);
    __syncthreads();
    sum_side_by_side(reinterpret_cast<float *>(smem), 4 * NB * blockDim.x, (int)p.D, part_out);
}

// ---- rows too long for registers: a CTA each, two passes (the second through L1 and L2)
template <typename E, bool WIDE>
__global__ void __launch_bounds__(kRowThreads) rms_fwd_kernel(RmsParams p) {
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
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
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
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

// Sums of dy hat over `parts` blocks of rows: a thread per column.
template <typename E>
__global__ void __launch_bounds__(128) rms_weight_part_kernel(RmsParams p, int parts, float *part) {
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    const int at = blockIdx.x % parts;
    const int64_t c = (int64_t)(blockIdx.x / parts) * 128 + threadIdx.x, each = ceil_div(p.rows, parts), r0 = at * each, r1 = min(r0 + each, p.rows);
    if (c >= p.D) return;
    const E *x = static_cast<const E *>(p.x) + c, *dy = static_cast<const E *>(p.dout) + c;
    float s = 0.f;
#pragma unroll 4
    for (int64_t row = r0; row < r1; ++row) s = fmaf(to_f(dy[row * p.ds]), to_f(x[row * p.xs]) * p.rstd[row], s);
    part[at * p.D + c] = s;
}

// 32 columns per CTA, the parts in 32 slices, in a fixed order.  (A slice's loads one after
// the other took 1.3 us more.)
__global__ void __launch_bounds__(1024) rms_weight_sum_kernel(RmsParams p, int64_t parts, const float *part) {
    constexpr int kAtOnce = 5;   // of 152 parts all
    sm103::wait_for_prior_kernels();
    sm103::allow_next_kernel();
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < p.D) {
        for (int64_t j = slice; j < parts; j += 32 * kAtOnce) {
            float f[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) f[i] = j + 32 * i < parts ? part[(j + 32 * i) * p.D + c] : 0.f;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) t += f[i];
        }
    }
    sums[slice][lane] = t;
    __syncthreads();
    t = sums[lane][slice];             // warp `slice` adds up column `slice`
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int64_t mine = (int64_t)blockIdx.x * 32 + slice;
    if (lane == 0 && mine < p.D) p.dweight[mine] = t;
}

// Groups of n elements where every row allows them.
bool aligned_rows(const RmsParams &p, int n, std::initializer_list<std::pair<const void *, int64_t>> tensors) {
    const size_t bytes = n * dtype_bytes(p.dtype);
    for (const auto &t : tensors)
        if (t.first && (reinterpret_cast<uintptr_t>(t.first) % bytes || t.second % n)) return false;
    return reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;
}
dim3 row_block(int64_t D, int el, int most) {
    const int x = (int)(ceil_div(D, 32 * el) * 32);
    return dim3(x, x >= most ? 1 : most / x);
}

constexpr int64_t kFwdMaxD = 16384;
int64_t bwd_most(const RmsParams &p) { return kBwdThreads * (p.dtype == kFP32 ? kBwdMost<float> : kBwdMost<__half>); }

bool fwd_in_registers(const RmsParams &p) {
    const int V = 16 / (int)dtype_bytes(p.dtype);
    return p.D <= kFwdMaxD && p.D % V == 0 && aligned_rows(p, V, {{p.x, p.xs}, {p.res, p.rs}, {p.res_out, p.ros}}) &&
           (p.out_dtype == p.dtype ? aligned_rows(p, V, {{p.out, p.os}})
                                   : reinterpret_cast<uintptr_t>(p.out) % V == 0 && p.os % V == 0);
}
bool bwd_in_registers(const RmsParams &p) {
    const int V = 16 / (int)dtype_bytes(p.dtype);
    return p.D <= bwd_most(p) && p.D % V == 0 && aligned_rows(p, V, {{p.x, p.xs}, {p.dout, p.ds}, {p.dres, p.drs}, {p.dx, p.D}});
}
// Elements per thread: a warp to a short row; many of longer ones, as each row costs a thread about
// 150 instructions beside those of its elements, but few where an SM has up to 4 rows (64 x 4096 bf16
// 5.6 us with 8, 7.6 with 32; 1200 x 4096 11.3 and 10.5).
int bwd_el(const RmsParams &p, int sms) {
    const int most = p.dtype == kFP32 ? kBwdMost<float> : kBwdMost<__half>;
    const bool few = p.rows <= 4 * sms;
    if (few && p.D <= 8192) return p.D <= 4096 ? 8 : 16;
    return p.D <= 256 ? 8 : p.D <= 512 || most == 16 ? 16 : 32;
}
// A few rows, up to `most` KB a tensor, are one cluster's or one CTA's, which have the whole gradient of
// the weight: no workspace and no second launch, which take the host 5 us (a call 13 us instead of 18).
// On the GPU, with a cluster and without: 64 x 256 bf16 2.7 us and 4.1, 64 x 1024 4.1 and 4.3, 128 x
// 1024 (256 KB) 5.6 and 4.5; unaligned 32 x 1023 4.5 and 5.1, 16 x 4095 (128 KB) 7.2 and 6.0.  Up to
// 4 KB one CTA is as fast (2 x 256 2.0 us, a cluster 3.5).
int few_ctas(const RmsParams &p, int most) {
    const int64_t bytes = p.rows * p.D * (int64_t)dtype_bytes(p.dtype);
    return !p.dweight || bytes > most << 10 ? 0 : bytes <= 4 << 10 ? 1 : (int)std::min(p.rows, (int64_t)kFewCtas);
}
constexpr int kFew = 256, kFewOdd = 128;
// Rows side by side have barriers of their own, of which a CTA has 15 beside the common one; no
// more of them than leaves every SM a row.
dim3 bwd_block(const RmsParams &p, int sms) {
    dim3 block = row_block(p.D, bwd_el(p, sms), kBwdThreads);
    if (block.x > 32) block.y = std::min(block.y, 15u);
    const int few = few_ctas(p, kFew);
    block.y = (unsigned)std::min((int64_t)block.y, std::max(ceil_div(p.rows, few ? few : sms), (int64_t)1));
    return block;
}
int64_t bwd_grid(const RmsParams &p, int sms) {
    const int few = few_ctas(p, kFew);
    return few ? few : std::min(ceil_div(p.rows, (int64_t)bwd_block(p, sms).y), (int64_t)sms);
}
// Rows that are not aligned: 4 blocks of 128 to a warp, 2 where few rows leave most of the GPU idle.
int odd_blocks(const RmsParams &p, int sms) { return p.D <= 2 * 128 || p.rows <= 4 * sms ? 2 : 4; }
dim3 odd_block(const RmsParams &p, int nb, int most) {
    const int x = 32 * (int)ceil_div(ceil_div(p.D, kFp8Block), nb);
    return dim3(x, x >= most ? 1 : most / x);
}
// Longer ones pass over a row twice: 8192 x 8191 bf16 to 8 bits takes 140 us so, and 270 us with 8
// blocks to a warp in registers, of which too few warps fit.
constexpr int64_t kOddFwdMaxD = 4096, kOddBwdMaxD = 8192;
// Backward: as many CTAs as the registers let an SM hold (16 warps)
dim3 odd_bwd_block(const RmsParams &p) { return odd_block(p, 4, 256); }
int64_t odd_bwd_grid(const RmsParams &p, int sms) {
    const dim3 block = odd_bwd_block(p);
    if (const int few = few_ctas(p, kFewOdd)) return few;
    return std::min(ceil_div(p.rows, (int64_t)block.y), (int64_t)sms * std::max(512 / (int)(block.x * block.y), 1));
}
int64_t weight_parts(const RmsParams &p, int sms) {
    if (p.rows == 0) return 0;
    if (bwd_in_registers(p)) return few_ctas(p, kFew) ? 1 : bwd_grid(p, sms);
    return p.D <= kOddBwdMaxD ? few_ctas(p, kFewOdd) ? 1 : odd_bwd_grid(p, sms) : std::min(ceil_div(p.rows, 64), (int64_t)256);
}

template <typename E, int NB>
cudaError_t run_fwd_odd(const RmsParams &p, cudaStream_t stream) {
    const dim3 block = odd_block(p, NB, 256);
    const auto run = [&](auto kernel) { return launch_early(kernel, ceil_div(p.rows, (int64_t)block.y), block, 0, stream, 0, p); };
    if (p.out_dtype == p.dtype) return run(rms_fwd_odd_kernel<E, NB, 0>);
    return p.out_dtype == kE4M3 ? run(rms_fwd_odd_kernel<E, NB, kE4M3>) : run(rms_fwd_odd_kernel<E, NB, kE5M2>);
}

template <typename E, int EL>
cudaError_t run_fwd(const RmsParams &p, cudaStream_t stream) {
    const dim3 block = row_block(p.D, EL, 256);
    const auto run = [&](auto kernel) { return launch_early(kernel, ceil_div(p.rows, (int64_t)block.y), block, 0, stream, 0, p); };
    if (p.out_dtype == p.dtype) return run(rms_fwd_row_kernel<E, EL, 0>);
    return p.out_dtype == kE4M3 ? run(rms_fwd_row_kernel<E, EL, kE4M3>) : run(rms_fwd_row_kernel<E, EL, kE5M2>);
}

template <typename E, int EL>
cudaError_t run_bwd(const RmsParams &p, float *part, int sms, cudaStream_t stream) {
    const dim3 block = bwd_block(p, sms);
    constexpr int kBytes = EL * 3 * kBwdStages<E, EL> * (int)sizeof(E);   // of a thread's ring
    constexpr auto kernel = rms_bwd_row_kernel<E, EL>;
    const cudaError_t e = allow_smem<kernel>(kBwdThreads * kBytes);
    if (e != cudaSuccess) return e;
    static_assert(kBytes >= EL * 4, "the sums fit the ring");
    const int few = few_ctas(p, kFew);
    return launch_early(kernel, bwd_grid(p, sms), block, block.x * block.y * kBytes, stream, few > 1 ? few : 0, p, part);
}

}  // namespace

size_t rms_bwd_scratch_bytes(const RmsParams &p, int sms) {
    const int64_t parts = p.dweight ? weight_parts(p, sms) : 0;
    return parts > 1 ? (size_t)(parts * p.D) * sizeof(float) : 0;
}

cudaError_t launch_rms_fwd(const RmsParams &p, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (fwd_in_registers(p)) {
            // elements per thread: a warp to a short row; of longer ones many, or few where few
            // rows leave most of the GPU idle
            if (p.D <= 256 || (p.rows <= 4 * sms && p.D <= 4096)) return run_fwd<E, 8>(p, stream);
            if (p.D <= 512 || (p.rows <= 4 * sms && p.D <= 8192)) return run_fwd<E, 16>(p, stream);
            return run_fwd<E, 32>(p, stream);
        }
        if (p.D <= kOddFwdMaxD) {
            return odd_blocks(p, sms) == 2 ? run_fwd_odd<E, 2>(p, stream) : run_fwd_odd<E, 4>(p, stream);
        }
        const bool wide = aligned_rows(p, 4, {{p.x, p.xs}, {p.res, p.rs}, {p.res_out, p.ros}}) &&
                          (p.out_dtype != p.dtype || aligned_rows(p, 4, {{p.out, p.os}}));
        return launch_early(wide ? rms_fwd_kernel<E, true> : rms_fwd_kernel<E, false>, p.rows, dim3(kRowThreads), 0, stream, 0, p);
    });
}

cudaError_t launch_rms_bwd(const RmsParams &p, unsigned char *ws, int sms, cudaStream_t stream) {
    const int64_t parts = weight_parts(p, sms);
    float *part = parts == 1 || !p.dweight ? p.dweight : reinterpret_cast<float *>(ws);
    const cudaError_t e = with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (p.rows == 0) return cudaSuccess;
        if (bwd_in_registers(p)) {
            const int el = bwd_el(p, sms);
            if (el == 8) return run_bwd<E, 8>(p, part, sms, stream);
            if (el == 16) return run_bwd<E, 16>(p, part, sms, stream);
            if constexpr (sizeof(E) == 2) return run_bwd<E, 32>(p, part, sms, stream);
        }
        if (p.D <= kOddBwdMaxD) {
            const dim3 block = odd_bwd_block(p);
            const int few = few_ctas(p, kFewOdd);
            return launch_early(rms_bwd_odd_kernel<E, 4>, odd_bwd_grid(p, sms), block, 16 * block.x * block.y * 4, stream, few > 1 ? few : 0, p, part);
        }
        const bool wide = aligned_rows(p, 4, {{p.x, p.xs}, {p.dout, p.ds}, {p.dres, p.drs}, {p.dx, p.D}});
        const cudaError_t e =
            launch_early(wide ? rms_bwd_kernel<E, true> : rms_bwd_kernel<E, false>, p.rows, dim3(kRowThreads), 0, stream, 0, p);
        if (e != cudaSuccess || !p.dweight) return e;
        return launch_early(rms_weight_part_kernel<E>, ceil_div(p.D, 128) * parts, dim3(128), 0, stream, 0, p, (int)parts, part);
    });
    if (e != cudaSuccess || part == p.dweight) return e;
    return launch_early(rms_weight_sum_kernel, ceil_div(p.D, 32), dim3(1024), 0, stream, 0, p, parts, part);
}

}  // namespace kda
