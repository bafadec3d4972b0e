// Gated linear recurrence, forward: h_t = a_t h_{t-1} + sigma(i_t) x_t per channel, a_t the
// gate's decay (glr_gate.cuh), h in fp32.
//
// One thread per (sequence, channel) walks its tokens; lanes hold neighbouring channels.
#include "glr_gate.cuh"

namespace kda {
namespace {

using namespace layer;

template <typename E, bool UB>
__global__ void __launch_bounds__(256) glr_fwd_serial_kernel(GlrParams p) {
    const int64_t unit = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (unit >= p.N * p.D) return;
    const int64_t n = unit / p.D, c = unit % p.D;
    int64_t lo, hi;
    seq_rows(p, n, lo, hi);
    const GateConst gc{expf(p.A_log[c / p.K]), p.dt_bias[c]};
    float h = p.init ? ld_state(p.init, p.state_type, unit) : 0.f;
    for (int64_t t = lo; t < hi; ++t) {
        if (p.checkpoints && t % kGlrCheckpointRows == 0) p.checkpoints[t / kGlrCheckpointRows * p.D + c] = h;
        const float x = to_f(static_cast<const E *>(p.x)[t * p.xs + c]);
        const float i = to_f(static_cast<const E *>(p.i)[t * p.is + c]);
        const float g = to_f(static_cast<const E *>(p.g)[t * p.gs + c]);
        h = gate_decay<UB>(g, gc, p.lower_bound) * h + sigmoid(i) * x;
        if (p.out) static_cast<E *>(p.out)[t * p.os + c] = from_f<E>(h);
    }
    if (p.fin) st_state(p.fin, p.state_type, unit, h);
}

}  // namespace

size_t glr_fwd_scratch_bytes(const GlrParams &, int) { return 0; }

cudaError_t launch_glr_fwd(const GlrParams &p, unsigned char *, int, cudaStream_t stream) {
    const unsigned grid = (unsigned)ceil_div(p.N * p.D, 256);
    with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (p.unbounded) glr_fwd_serial_kernel<E, true><<<grid, 256, 0, stream>>>(p);
        else glr_fwd_serial_kernel<E, false><<<grid, 256, 0, stream>>>(p);
    });
    return cudaGetLastError();
}

}  // namespace kda
