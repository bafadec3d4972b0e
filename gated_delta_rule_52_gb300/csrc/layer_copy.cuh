// Asynchronous copies into a thread's own slots of shared memory, and sums of partial
// results over CTAs.
#pragma once

#include "kda_chunk.cuh"
#include "layer_io.cuh"
#include "sm103.cuh"

namespace kda {
namespace layer {

// Copies n bytes (4, 8 or 16) of one thread.
template <int n>
__device__ __forceinline__ void copy_async(void *slot, const void *src) {
    static_assert(n == 4 || n == 8 || n == 16, "copy size");
    if constexpr (n == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm103::smem_u32(slot)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(sm103::smem_u32(slot)), "l"(src), "n"(n) : "memory");
}
// What a thread's slot holds of a row: its V elements, or the 4-byte words around V 16-bit
// elements whose row may begin inside a word.
template <int N>
struct Words { uint32_t w[N]; };
template <typename E, int V, bool WIDE>
using RowSlot = std::conditional_t<WIDE || sizeof(E) == 4, Pack<E, V>, Words<V / 2 + 1>>;
// Copies `count` <= N groups of V elements, `stride` elements apart, into slots THREADS
// groups apart.  WIDE: every group is aligned to its size and whole.  Else its first `cols`
// <= V elements are copied: 4-byte ones one by one, 2-byte ones, which have no asynchronous
// copy, as words, the last one no further than the elements go.  (Loaded and stored one by
// one they held up every group of rows: the convolution of 16384 x 4095 bf16 took 183 us
// forward and, of 8192 x 4095, 240 us backward; with words 100 us both.)
template <typename E, int V, bool WIDE, int N, int THREADS>
__device__ __forceinline__ void copy_rows(RowSlot<E, V, WIDE> *slots, const E *src, int64_t stride, int count, int cols) {
    if constexpr (WIDE) {
        if (count >= N) {
#pragma unroll
            for (int r = 0; r < N; ++r, src += stride) copy_async<sizeof(E) * V>(slots + r * THREADS, src);
        } else {
#pragma unroll 1
            for (int r = 0; r < count; ++r, src += stride) copy_async<sizeof(E) * V>(slots + r * THREADS, src);
        }
    } else if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int r = 0; r < N; ++r, src += stride) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (r < count && v < cols) copy_async<4>(&slots[r * THREADS].e[v], src + v);
        }
    } else {
#pragma unroll
        for (int r = 0; r < N; ++r, src += stride) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(src), word = at & ~(uintptr_t)3;
            const int bytes = 2 * cols + (int)(at & 2);
#pragma unroll
            for (int k = 0; k < V / 2 + 1; ++k)
                if (r < count && 4 * k < bytes)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sm103::smem_u32(&slots[r * THREADS].w[k])),
                                 "l"(word + 4 * k), "r"(min(bytes - 4 * k, 4))
                                 : "memory");
        }
    }
}
// The elements of a slot; `odd`: its row begins in the middle of a word.
template <typename E, int V>
__device__ __forceinline__ void take(const Pack<E, V> &slot, int, float (&f)[V]) { unpack<E, V>(slot, f); }
template <typename E, int V>
__device__ __forceinline__ void take(const Words<V / 2 + 1> &slot, int odd, float (&f)[V]) {
    Pack<E, V> t;
#pragma unroll
    for (int k = 0; k < V / 2; ++k) reinterpret_cast<uint32_t *>(t.e)[k] = __funnelshift_r(slot.w[k], slot.w[k + 1], 16 * odd);
    unpack<E, V>(t, f);
}
// Whether the rows of 16-bit elements from p on begin in the middle of a word.
struct RowParity {
    int first, step;
    __device__ __forceinline__ RowParity(const void *p, int64_t stride) : first((int)(reinterpret_cast<uintptr_t>(p) >> 1 & 1)), step((int)(stride & 1)) {}
    __device__ __forceinline__ int operator[](int r) const { return first ^ (step & r & 1); }
};
// Stores V values, or the first `cols` of them one by one.
template <typename E, int V, bool WIDE>
__device__ __forceinline__ void st_cols(E *p, const float (&f)[V], int cols) {
    if constexpr (WIDE) {
        st_f<E, V>(p, f);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < cols) p[v] = from_f<E>(f[v]);
    }
}
template <typename E, int V, bool WIDE>
__device__ __forceinline__ void ld_cols(const E *p, float (&f)[V], int cols) {
    if constexpr (WIDE) {
        ld_f<E, V>(p, f);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = v < cols ? to_f(p[v]) : 0.f;
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Tensor maps of token tensors [rows, D]: boxes of `box_rows` rows by `box_cols` channels,
// dense in shared memory, zeros where the tensor has no elements.
__device__ __forceinline__ void tma_box(void *dst, const CUtensorMap &map, uint64_t *bar, int c, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            sm103::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(&map)), "r"(sm103::smem_u32(bar)), "r"(c), "r"(row)
        : "memory");
}

// A tensor map's demands: 16-byte aligned rows, no row over another.
inline bool tma_rows(const void *ptr, int64_t stride, int64_t D, size_t elem) {
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && stride * elem % 16 == 0 && D * elem % 16 == 0 && stride >= D;
}
inline bool encode_tile_map(CUtensorMap &map, const void *ptr, int64_t stride, int64_t rows, int64_t D, int dtype, int box_cols,
                            int box_rows) {
    const auto encode = chunk::encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * dtype_bytes(dtype)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, step[2] = {1, 1};
    const CUtensorMapDataType type = dtype == kBF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : dtype == kFP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    return encode(&map, type, 2, const_cast<void *>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Lets a kernel use this much dynamic shared memory; set once per device.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<bool> done[kMaxDevices];
    return once_per_device(done, [&](int) { return cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}

// Launches a kernel that may start while the one before it on the stream ends.  The kernel calls
// sm103::wait_for_prior_kernels() before it touches global memory: everything up to there, and the
// way to the GPU, costs nothing then.  (A product in a row of them: 2 us less of 16.)
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), int64_t grid, dim3 block, size_t smem, cudaStream_t stream, int cluster, const Args &...args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = cluster > 0 ? 2 : 1;   // 0: no clusters
    return cudaLaunchKernelEx(&c, kernel, Params(args)...);
}

// Sum over j of part[j * width + c], 32 columns per CTA of kSumThreads threads, in a fixed
// order.  The threads of the CTA's first warp have the sum of column 32 blockIdx.x + lane.
constexpr int kSumThreads = 256;
__device__ __forceinline__ float column_sum(const float *part, int64_t parts, int64_t width, int64_t c, bool in) {
    constexpr int kSlices = kSumThreads / 32;
    __shared__ float sums[kSlices][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    float t = 0.f;
    if (in) {
#pragma unroll 8
        for (int64_t j = slice; j < parts; j += kSlices) t += part[j * width + c];
    }
    sums[slice][lane] = t;
    __syncthreads();
    t = 0.f;
#pragma unroll
    for (int j = 0; j < kSlices; ++j) t += sums[j][lane];
    return t;
}

}  // namespace layer
}  // namespace kda
