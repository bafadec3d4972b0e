// Gated linear recurrence, backward.  With e_t the gradient of h_t,
//   e_t = dout_t + a_{t+1} e_{t+1}   (e of the last token also takes dfinal)
//   dx = e s, di = e x s (1 - s), s = sigma(i);   dl = e_t a_t h_{t-1}, the gradient of gk_t;
//   dg = dl d gk/dg, ddt_bias = sum dg, dA_log = sum dl d gk/dA_log, dinit = a_first e_first.
// h_{t-1} is recomputed in fp32 from the checkpoints (one state every 64 packed rows).
//
// One thread per (sequence, channel) walks its 64-row blocks from the last to the first.
#include "glr_gate.cuh"

namespace kda {
namespace {

using namespace layer;

template <typename E, bool UB>
__global__ void __launch_bounds__(256) glr_bwd_serial_kernel(GlrParams p, float *dA_part, float *ddt_part) {
    const int64_t unit = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (unit >= p.N * p.D) return;
    const int64_t n = unit / p.D, c = unit % p.D;
    int64_t lo, hi;
    seq_rows(p, n, lo, hi);
    const GateConst gc = gate_const<UB>(p.A_log[c / p.K], p.dt_bias[c]);
    const float lb2 = p.lower_bound * kLog2e;
    const E *xp = static_cast<const E *>(p.x), *ip = static_cast<const E *>(p.i), *gp = static_cast<const E *>(p.g);
    float e = p.dfinal ? p.dfinal[unit] : 0.f, dA_sum = 0.f, ddt_sum = 0.f;
    float start[kGlrCheckpointRows];
    for (int64_t end = hi; end > lo;) {
        const int64_t begin = max(lo, (end - 1) / kGlrCheckpointRows * kGlrCheckpointRows);
        float h = begin % kGlrCheckpointRows == 0 ? p.checkpoints[begin / kGlrCheckpointRows * p.D + c]
                  : p.init                        ? ld_state(p.init, p.state_type, unit)
                                                  : 0.f;
        for (int64_t t = begin; t < end; ++t) {
            start[t - begin] = h;
            h = gate_decay<UB>(to_f(gp[t * p.gs + c]), gc, lb2) * h + sigmoid(to_f(ip[t * p.is + c])) * to_f(xp[t * p.xs + c]);
        }
        for (int64_t t = end - 1; t >= begin; --t) {
            const float x = to_f(xp[t * p.xs + c]);
            float slope, rate, s, ss;
            const float a = gate_slopes<UB>(to_f(gp[t * p.gs + c]), gc, lb2, slope, rate);
            sigmoid_slope(to_f(ip[t * p.is + c]), s, ss);
            e += to_f(static_cast<const E *>(p.dout)[t * p.ds + c]);
            const float dl = e * a * start[t - begin], dg = dl * slope;
            static_cast<E *>(p.dx)[t * p.D + c] = from_f<E>(e * s);
            static_cast<E *>(p.di)[t * p.D + c] = from_f<E>(e * x * ss);
            static_cast<E *>(p.dg)[t * p.D + c] = from_f<E>(dg);
            ddt_sum += dg;
            dA_sum += dl * rate;
            e *= a;
        }
        end = begin;
    }
    if (p.dinit) p.dinit[unit] = e;
    dA_part[unit] = dA_sum;
    ddt_part[unit] = ddt_sum;
}

// Sums the partial parameter gradients [parts, D]: ddt_bias per channel, dA_log per head.
__global__ void __launch_bounds__(256) glr_param_grads_kernel(GlrParams p, int64_t parts, const float *dA_part,
                                                              const float *ddt_part) {
    __shared__ float sums[256];
    const int64_t h = blockIdx.x;
    float dA = 0.f;
    for (int64_t k = threadIdx.x; k < p.K; k += 256) {
        const int64_t c = h * p.K + k;
        float ddt = 0.f;
        for (int64_t j = 0; j < parts; ++j) {
            ddt += ddt_part[j * p.D + c];
            dA += dA_part[j * p.D + c];
        }
        p.ddt_bias[c] = ddt;
    }
    sums[threadIdx.x] = dA;
    __syncthreads();
    for (int w = 128; w; w >>= 1) {
        if (threadIdx.x < w) sums[threadIdx.x] += sums[threadIdx.x + w];
        __syncthreads();
    }
    if (threadIdx.x == 0) p.dA_log[h] = sums[0];
}

// The forward run that writes checkpoints only.
GlrParams states_only(const GlrParams &p) {
    GlrParams f = p;
    f.out = f.fin = nullptr;
    return f;
}

}  // namespace

size_t glr_bwd_scratch_bytes(const GlrParams &p, int sms) {
    const size_t part = (size_t)(p.N * p.D) * sizeof(float);
    const size_t ck = p.checkpoints ? 0 : (size_t)(ceil_div(p.rows, kGlrCheckpointRows) * p.D) * sizeof(float);
    return (2 * part + ck + 15) / 16 * 16 + (p.checkpoints ? 0 : glr_fwd_scratch_bytes(states_only(p), sms));
}

cudaError_t launch_glr_bwd(const GlrParams &p0, unsigned char *ws, int sms, cudaStream_t stream) {
    GlrParams p = p0;
    const int64_t units = p.N * p.D;
    float *dA_part = reinterpret_cast<float *>(ws), *ddt_part = dA_part + units;
    if (units > 0) {
        if (!p.checkpoints) {
            p.checkpoints = ddt_part + units;
            const size_t used = (size_t)(2 * units + ceil_div(p.rows, kGlrCheckpointRows) * p.D) * sizeof(float);
            const cudaError_t e = launch_glr_fwd(states_only(p), ws + (used + 15) / 16 * 16, sms, stream);
            if (e != cudaSuccess) return e;
        }
        const unsigned grid = (unsigned)ceil_div(units, 256);
        with_dtype(p.dtype, [&](auto *tag) {
            using E = std::remove_pointer_t<decltype(tag)>;
            if (p.unbounded) glr_bwd_serial_kernel<E, true><<<grid, 256, 0, stream>>>(p, dA_part, ddt_part);
            else glr_bwd_serial_kernel<E, false><<<grid, 256, 0, stream>>>(p, dA_part, ddt_part);
        });
    }
    glr_param_grads_kernel<<<(unsigned)p.H, 256, 0, stream>>>(p, p.N, dA_part, ddt_part);
    return cudaGetLastError();
}

}  // namespace kda
