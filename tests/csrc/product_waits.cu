// The bounded waits of the 8-bit product (csrc/fp8_mm.cu), by a warp, on a barrier with `arrivals` of the
// one arrival that completes its phase.
#include "../../gated_delta_rule_52_gb300/csrc/fp8_mm.cu"

namespace kda {
namespace {

template <bool CLUSTER>
__global__ void barrier_wait(int arrivals, uint64_t limit, int *got) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncwarp();
    if (threadIdx.x == 0 && arrivals) mbar_arrive(&bar);
    const bool ok = warp_wait<CLUSTER>(&bar, 0, limit);
    got[threadIdx.x] = ok;
}

}  // namespace
}  // namespace kda

extern "C" int product_wait(int cluster, int arrivals, uint64_t limit_ns, int *got, cudaStream_t stream) {
    if (cluster) kda::barrier_wait<true><<<1, 32, 0, stream>>>(arrivals, limit_ns, got);
    else kda::barrier_wait<false><<<1, 32, 0, stream>>>(arrivals, limit_ns, got);
    return (int)cudaGetLastError();
}
extern "C" uint64_t product_wait_limit() { return kda::kWait; }
