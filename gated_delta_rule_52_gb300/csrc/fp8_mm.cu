// Product of 8-bit tensors with a power-of-two scale for each block of 128 along K:
//   out[m, n] = add[m, n] + sum over blocks j of 2^(ea[m, j] + eb[n, j]) sum over k in j of a[m, k] b[n, k]
// The tensor cores multiply the scales in (block-scaled tcgen05.mma), so that one fp32
// accumulator in TMEM takes all of K.  The MMA has a scale per 32 elements of K; 4 MMAs of a
// block take the same byte.  4 blocks' bytes of a row are one 4-byte word, the unit in which
// scales are loaded and put into TMEM.
#include <algorithm>
#include <cuda.h>

#include "kda_chunk.cuh"
#include "layer_copy.cuh"
#include "layer_io.cuh"
#include "sm103.cuh"

namespace kda {
namespace {

using namespace layer;
using namespace sm103;

constexpr uint64_t kWait = 2000000000ull;   // 2 s per wait
constexpr int kRows = 128;                  // rows of b per tile: the MMA's M, TMEM's lanes
constexpr int kScaleStages = 4;

struct MatmulArgs {
    CUtensorMap a, b;
    MatmulParams p;
};

__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap &map, uint64_t *bar, int k, int row) {
    tma_box(dst, map, bar, k, row);
}

// Asynchronous copy of up to 4 bytes (the rest zero) into shared memory.
__device__ __forceinline__ void copy_word(uint32_t dst, const uint8_t *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The scale words of rows row0 .. row0 + n (of blocks 4 group .. 4 group + 3) to `dst`, as the
// tensor cores want them: rows 128 c + 32 w + i at byte 512 c + 16 i + 4 w.
__device__ __forceinline__ void copy_scales(uint32_t dst, const Fp8Operand &o, int64_t row0, int n, int group, int blocks, int lane) {
    const int bytes = min(4, blocks - 4 * group);
    for (int r = lane; r < n; r += 32) {
        const int64_t row = row0 + r;
        const bool in = row < o.rows;
        const uint8_t *src = o.s + (in ? (o.tile ? row / kFp8Block : row) * o.s_stride + 4 * group : 0);
        copy_word(dst + (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4, src, in ? bytes : 0);
    }
}

// ---- one tile of 128 rows of b by BT rows of a per cluster of `split` CTAs, which share K and
// join their sums through distributed shared memory.
template <int BT>
struct TileShape {
    static constexpr int kStage = (kRows + BT) * kFp8Block;
    static constexpr int kStages = BT <= 16 ? 6 : BT <= 32 ? 5 : BT <= 64 ? 4 : BT <= 128 ? 3 : 4;
    static constexpr int kScaleA = BT <= 128 ? 512 : 1024;
    static constexpr int kScaleStage = 512 + kScaleA;
    static constexpr int kSmem = 1024 + kStage * kStages + kScaleStage * kScaleStages;
    // TMEM columns: the accumulator, and two sets of scales
    static constexpr int kSet = 4 + kScaleA / 128;
    static constexpr int kCols = BT + 2 * kSet <= 32 ? 32 : BT + 2 * kSet <= 64 ? 64 : BT + 2 * kSet <= 128 ? 128 : BT + 2 * kSet <= 256 ? 256 : 512;
    static_assert(BT * kRows * 4 <= kStage * kStages, "the sums fit the ring");
};

template <typename E, int BT>
__global__ void __launch_bounds__(128) mm_tile_kernel(const __grid_constant__ MatmulArgs args, int split) {
    using S = TileShape<BT>;
    extern __shared__ unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char *scales = ring + S::kStage * S::kStages;
    __shared__ uint64_t full[S::kStages], empty[S::kStages], sfull[kScaleStages], sempty[kScaleStages], done;
    __shared__ uint32_t tmem_base;
    const MatmulParams &p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % split;
    const int64_t tile = blockIdx.x / split, across = ceil_div(p.b.rows, kRows), m0 = tile / across * BT, n0 = tile % across * kRows;
    const int blocks = (int)ceil_div(p.K, kFp8Block);
    const int k0 = (int)((int64_t)blocks * rank / split), k1 = (int)((int64_t)blocks * (rank + 1) / split);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < kScaleStages; ++i) mbar_init(&sfull[i], 32), mbar_init(&sempty[i], 1);
        mbar_init(&done, 1);
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(&tmem_base, S::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t acc = tmem_base, sf = acc + BT;
    bool ok = true;
    if (warp == 0 && lane == 0) {
        int i = 0;
        for (int k = k0; k < k1; ++k, ++i) {
            const int st = i % S::kStages, turn = i / S::kStages;
            if (turn > 0 && !mbar_wait(&empty[st], (turn - 1) & 1, kWait)) {
                ok = false;
                break;
            }
            unsigned char *at = ring + st * S::kStage;
            mbar_arrive_expect_tx(&full[st], S::kStage);
            tma_tile(at, args.b, &full[st], k * kFp8Block, (int)n0);
            tma_tile(at + kRows * kFp8Block, args.a, &full[st], k * kFp8Block, (int)m0);
        }
        // the copies end before the CTA does
        for (int j = max(0, i - S::kStages); j < i; ++j)
            if (!mbar_wait(&full[j % S::kStages], (j / S::kStages) & 1, kWait)) ok = false;
    } else if (warp == 1 && lane == 0) {
        int i = 0, g = -1, sets = 0;
        for (int k = k0; ok && k < k1; ++k, ++i) {
            const int st = i % S::kStages;
            if (k / 4 != g) {
                g = k / 4;
                const int ss = sets % kScaleStages;
                if (!mbar_wait(&sfull[ss], (sets / kScaleStages) & 1, kWait)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t from = smem_u32(scales + ss * S::kScaleStage), to = sf + (sets & 1) * S::kSet;
                tmem_copy_scales(to, sdesc_plain(from, 128));
                for (int c = 0; c < S::kScaleA / 512; ++c) tmem_copy_scales(to + 4 + 4 * c, sdesc_plain(from + 512 + 512 * c, 128));
                mma_commit(&sempty[ss]);
                ++sets;
            }
            if (!mbar_wait(&full[st], (i / S::kStages) & 1, kWait)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t set = sf + ((sets - 1) & 1) * S::kSet, at = smem_u32(ring + st * S::kStage);
            const uint32_t idesc = idesc_mx8(kRows, BT, p.b.dtype == kE5M2, p.a.dtype == kE5M2, k & 3);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                mma_mx8(acc, sdesc_sw128(at + 32 * q, 16, 1024), sdesc_sw128(at + kRows * kFp8Block + 32 * q, 16, 1024), idesc, set,
                        set + 4, i > 0 || q > 0);
            mma_commit(&empty[st]);
        }
        mma_commit(&done);
    } else if (warp == 2) {
        // kScaleStages - 1 groups on their way; a group is handed over when the copies before
        // the last kScaleStages - 2 have arrived
        const int g0 = k0 / 4, groups = k1 > k0 ? (k1 - 1) / 4 - g0 + 1 : 0;
        constexpr int kAhead = kScaleStages - 2;
        for (int i = 0; i < groups + kAhead; ++i) {
            if (i < groups) {
                const int ss = i % kScaleStages, turn = i / kScaleStages;
                if (turn > 0 && !mbar_wait(&sempty[ss], (turn - 1) & 1, kWait)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t at = smem_u32(scales + ss * S::kScaleStage);
                copy_scales(at, p.b, n0, kRows, g0 + i, blocks, lane);
                copy_scales(at + 512, p.a, m0, BT, g0 + i, blocks, lane);
            }
            copies_commit();
            if (i >= kAhead) {
                copies_wait<kAhead>();
                fence_proxy_async_smem();
                mbar_arrive(&sfull[(i - kAhead) % kScaleStages]);
            }
        }
        copies_wait<0>();
    }
    __syncwarp();
    if (!mbar_wait(&done, 0, 2 * kWait)) ok = false;
    if (!ok && p.err) atomicExch(p.err, kErrTimeout);
    __syncthreads();   // the ring is free: every copy and MMA has ended
    tc_fence_after();
    // sums to shared memory, [BT][128]
    float *sums = reinterpret_cast<float *>(ring);
    for (int c = 0; c < BT; c += 16) {
        float r[16];
        if (k1 > k0) {
            tmem_ld16(tmem_addr(acc, warp * 32, c), r);
            tmem_ld_wait();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) sums[(c + j) * kRows + threadIdx.x] = k1 > k0 ? r[j] : 0.f;
    }
    tc_fence_before();
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp == 3) tmem_dealloc(acc, S::kCols);
    // each CTA's part of the tile's rows of a
    const int c0 = BT * rank / split, c1 = BT * (rank + 1) / split;
    const int64_t n = n0 + threadIdx.x;
    const uint32_t mine = smem_u32(sums);
    for (int c = c0; c < c1; ++c) {
        const int64_t m = m0 + c;
        if (m >= p.a.rows) break;
        float t = 0.f;
        if (split == 1) {
            t = sums[c * kRows + threadIdx.x];
        } else {
            for (int q = 0; q < split; ++q) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(mine + (c * kRows + threadIdx.x) * 4, q)) : "memory");
                t += v;
            }
        }
        if (n < p.b.rows) {
            if (p.add) t += to_f(static_cast<const E *>(p.add)[m * p.as + n]);
            static_cast<E *>(p.out)[m * p.os + n] = from_f<E>(t);
        }
    }
    if (split > 1) cluster_sync();   // the others have read this CTA's sums
}

bool encode_operand(CUtensorMap &map, const Fp8Operand &o, int64_t K, int box_rows) {
    const auto encode = chunk::encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)o.rows}, strides[1] = {(cuuint64_t)o.stride};
    const cuuint32_t box[2] = {kFp8Block, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(o.q), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename E, int BT>
cudaError_t run_tile(MatmulArgs &args, int split, cudaStream_t stream) {
    using S = TileShape<BT>;
    constexpr auto kernel = mm_tile_kernel<E, BT>;
    cudaError_t e = allow_smem<kernel>(S::kSmem);
    if (e != cudaSuccess) return e;
    if (!encode_operand(args.a, args.p.a, args.p.K, BT)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(ceil_div(args.p.b.rows, kRows) * ceil_div(args.p.a.rows, BT) * split));
    c.blockDim = dim3(128);
    c.dynamicSmemBytes = S::kSmem;
    c.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = split, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args, split);
}

// out = add, where K is 0.
template <typename E>
__global__ void __launch_bounds__(256) mm_add_kernel(MatmulParams p) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.a.rows * p.b.rows; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / p.b.rows, n = i % p.b.rows;
        static_cast<E *>(p.out)[m * p.os + n] = p.add ? static_cast<const E *>(p.add)[m * p.as + n] : from_f<E>(0.f);
    }
}

}  // namespace

cudaError_t launch_matmul(const MatmulParams &p, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (p.K == 0) {
            mm_add_kernel<E><<<(unsigned)std::min(ceil_div(p.a.rows * p.b.rows, 256), (int64_t)sms * 8), 256, 0, stream>>>(p);
            return cudaGetLastError();
        }
        MatmulArgs args;
        args.p = p;
        if (!encode_operand(args.b, p.b, p.K, kRows)) return cudaErrorInvalidValue;
        const int64_t M = p.a.rows, tiles = ceil_div(p.b.rows, kRows), blocks = ceil_div(p.K, kFp8Block);
        const int bt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
        const int64_t all = tiles * ceil_div(M, bt);
        int split = 1;
        while (split < 8 && all * split < sms && blocks >= 8 * split) split *= 2;
        switch (bt) {
            case 16: return run_tile<E, 16>(args, split, stream);
            case 32: return run_tile<E, 32>(args, split, stream);
            case 64: return run_tile<E, 64>(args, split, stream);
            case 128: return run_tile<E, 128>(args, split, stream);
            default: return run_tile<E, 256>(args, split, stream);
        }
    });
}

}  // namespace kda
