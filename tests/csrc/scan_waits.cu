// The bounded waits of the gated linear recurrence's scans (csrc/glr_scan.cuh), each on
// something that never comes: `count` waits one after the other by one thread.
#include "../../gated_delta_rule_52_gb300/csrc/glr_scan.cuh"

namespace {

using namespace kda::layer;

__global__ void value_waits(const uint64_t *maps, const uint32_t *states, int count, int *err) {
    __shared__ int late;
    const Waits w{err, &late};
    late = 0;
    for (int k = 0; k < count; ++k) {
        await(w, states + k, peek(states + k));
        join_maps(maps + k, 1, 1, w);
    }
}

__global__ void copy_waits(int count, int *err) {
    __shared__ uint64_t arrived;
    __shared__ int late;
    kda::sm103::mbar_init(&arrived, 1);
    kda::sm103::fence_mbar_init();
    late = 0;
    for (int k = 0; k < count; ++k) wait_copies(&arrived, 0, {err, &late});
}

}  // namespace

extern "C" int scan_value_waits(const uint64_t *maps, const uint32_t *states, int count, int *err, cudaStream_t stream) {
    value_waits<<<1, 1, 0, stream>>>(maps, states, count, err);
    return (int)cudaGetLastError();
}
extern "C" int scan_copy_waits(int count, int *err, cudaStream_t stream) {
    copy_waits<<<1, 1, 0, stream>>>(count, err);
    return (int)cudaGetLastError();
}
