// Product of 8-bit tensors with a power-of-two scale for each block of 128 along K:
//   out[m, n] = add[m, n] + sum over blocks j of 2^(ea[m, j] + eb[n, j]) sum over k in j of a[m, k] b[n, k]
// The tensor cores multiply the scales in (block-scaled tcgen05.mma), so that one fp32
// accumulator in TMEM takes all of K.  The MMA has a scale per 32 elements of K; 4 MMAs of a
// block take the same byte.  4 blocks' bytes of a row are one 4-byte word, the unit in which
// scales are loaded and put into TMEM.
#include <algorithm>
#include <cstdlib>
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
constexpr int kScaleStages = 8, kAhead = 4;   // groups of 4 blocks' scales: places, and on their way

// Waits of the pipelines.  Reading the GPU's timer takes longer than a stage does, so it is read
// once in many tries only.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, uint64_t limit = kWait) {
    uint64_t t0 = 0;
    for (uint32_t tries = 0;; ++tries) {
        if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if (tries % 1024 == 1023) {
            const uint64_t now = globaltimer_ns();
            if (!t0) t0 = now;
            else if (now - t0 > limit) return false;
        }
    }
}

// wait_for by a whole warp.
template <bool CLUSTER>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t limit = kWait) {
    return __all_sync(0xffffffffu, wait_for<CLUSTER>(bar, parity, limit));
}

// A place in a ring of N slots and the parity of its turn.
template <int N>
struct Slot {
    int at = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) at = 0, turn ^= 1;
    }
};

struct MatmulArgs {
    CUtensorMap a, b, out;
    MatmulParams p;
};

__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap &map, uint64_t *bar, int k, int row) {
    tma_box(dst, map, bar, k, row);
}

// Asynchronous copy of up to 4 bytes (the rest zero) into shared memory.
__device__ __forceinline__ void copy_word(uint32_t dst, const uint8_t *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Scale words of N rows from row0 on, 4 blocks of K at a time, on their way to shared memory as the
// tensor cores want them: rows 128 c + 32 w + i at byte 512 c + 16 i + 4 w.  A lane has rows i =
// lane of every c and w; where they are is worked out once for a tile.
template <int N>
struct ScaleRows {
    static constexpr int kWords = (N + 31) / 32;
    const uint8_t *row[kWords];
    uint32_t in;   // which of them exist
    __device__ __forceinline__ void set(const Fp8Operand &o, int64_t row0, int lane) {
        in = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int64_t r = row0 + 32 * w + lane;
            const bool some = 32 * w + lane < N && r < o.rows;
            row[w] = o.s + (some ? (o.tile ? r / kFp8Block : r) * o.s_stride : 0);
            in |= (uint32_t)some << w;
        }
    }
    // The next 4 blocks, `bytes` (1 to 4) of which there are.
    __device__ __forceinline__ void copy(uint32_t dst, int bytes, int lane) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            copy_word(dst + (w >> 2) * 512 + lane * 16 + (w & 3) * 4, row[w], in >> w & 1 ? bytes : 0);
            if (in >> w & 1) row[w] += 4;
        }
    }
};

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
            if (turn > 0 && !wait_for<false>(&empty[st], (turn - 1) & 1)) {
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
            if (!wait_for<false>(&full[j % S::kStages], (j / S::kStages) & 1)) ok = false;
    } else if (warp == 1 && lane == 0) {
        int i = 0, g = -1, sets = 0;
        for (int k = k0; ok && k < k1; ++k, ++i) {
            const int st = i % S::kStages;
            if (k / 4 != g) {
                g = k / 4;
                const int ss = sets % kScaleStages;
                if (!wait_for<false>(&sfull[ss], (sets / kScaleStages) & 1)) {
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
            if (!wait_for<false>(&full[st], (i / S::kStages) & 1)) {
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
        // kAhead groups on their way while the ones before are handed over
        const int g0 = k0 / 4, groups = k1 > k0 ? (k1 - 1) / 4 - g0 + 1 : 0;
        ScaleRows<kRows> rows_b;
        ScaleRows<BT> rows_a;
        rows_b.set(p.b, n0, lane);
        rows_a.set(p.a, m0, lane);
#pragma unroll
        for (int w = 0; w < rows_b.kWords; ++w) rows_b.row[w] += rows_b.in >> w & 1 ? 4 * g0 : 0;
#pragma unroll
        for (int w = 0; w < rows_a.kWords; ++w) rows_a.row[w] += rows_a.in >> w & 1 ? 4 * g0 : 0;
        for (int i = 0; i < groups + kAhead; ++i) {
            if (i < groups) {
                const int ss = i % kScaleStages, turn = i / kScaleStages;
                if (turn > 0 && !wait_for<false>(&sempty[ss], (turn - 1) & 1)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t at = smem_u32(scales + ss * S::kScaleStage);
                const int bytes = min(4, blocks - 4 * (g0 + i));
                rows_b.copy(at, bytes, lane);
                rows_a.copy(at + 512, bytes, lane);
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
    if (!wait_for<false>(&done, 0, 2 * kWait)) ok = false;
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

// ---- tiles of 256 rows of a by BN rows of b, persistent pairs of CTAs.
//
// A pair shares its tiles: each CTA loads its 128 rows of a and half of the rows of b, one
// thread of the first CTA issues the MMAs of both (cta_group::2), which halves what shared
// memory has to deliver for b.  Warp 0 loads tiles, warp 2 scales, warp 1 issues, warps 4 to 11
// empty the accumulators; two of these in TMEM, so that a tile's MMAs run while the one before
// is stored.  fp32 outputs take K in segments whose sums are added in registers: the tensor
// cores cut an accumulator at each step, which over a long K would cost more than fp32's own
// rounding.
constexpr int kPairThreads = 384, kStoreWarps = 8;
constexpr int kSegment = 32;                // blocks of K per segment of an fp32 output

// A store warp's buffer: 32 rows of 64 bytes for a tensor store, or 32 x 17 fp32.
constexpr int kStoreBuffer = 2560;

template <int BN>
struct PairShape {
    static constexpr int kStage = (kRows + BN / 2) * kFp8Block;
    static constexpr int kScaleB = BN <= 128 ? 512 : 1024;
    static constexpr int kScaleStage = 512 + kScaleB;
    static constexpr int kStaging = kStoreWarps * kStoreBuffer;
    static constexpr int kStages = (227 * 1024 - 2048 - kStaging - kScaleStage * kScaleStages) / kStage;
    static constexpr int kSmem = 1024 + kStage * kStages + kScaleStage * kScaleStages + kStaging;
    static constexpr int kSet = 4 + kScaleB / 128;
    static constexpr int kBuffers = 2 * BN + 2 * kSet <= 512 ? 2 : 1;
    static constexpr int kCols = kBuffers * BN + 2 * kSet <= 256 ? 256 : 512;
    static_assert(kSmem <= 227 * 1024 && BN % 32 == 0 && kBuffers * BN + 2 * kSet <= 512, "fits an SM");
};

// Tile t of a grid of `down` x `across`: 8 tiles down, then across, so that the tiles in flight
// share rows of both operands in L2.
__device__ __forceinline__ void tile_at(int64_t t, int64_t down, int64_t across, int64_t &i, int64_t &j) {
    const int64_t band = t / (8 * across), first = band * 8, high = min(down - first, (int64_t)8), in = t - band * 8 * across;
    i = first + in % high;
    j = in / high;
}

// The first n of V neighbours (the others 0), in one load where all exist.
template <typename E, int V>
__device__ __forceinline__ Pack<E, V> ld_row(const E *p, int n) {
    if (n >= V) return ld_pack<E, V>(p);
    Pack<E, V> r;
#pragma unroll
    for (int e = 0; e < V; ++e) r.e[e] = e < n ? p[e] : from_f<E>(0.f);
    return r;
}

// 16 columns of 32 rows (one to a lane) to out, with the addend, by single elements: neighbouring
// lanes take neighbouring columns.  `own`: 32 x 17 fp32 of shared memory.
template <typename E>
__device__ __forceinline__ void st_narrow(const MatmulParams &p, const float (&r)[16], float *own, int64_t m0, int64_t n0, int lane) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) own[lane * 17 + e] = r[e];
    __syncwarp();
    const int64_t n = n0 + (lane & 15), m = m0 + (lane >> 4);
    const int rows = n < p.b.rows ? (int)min(max(p.a.rows - m, (int64_t)0), (int64_t)32) : 0;
    E *to = static_cast<E *>(p.out) + m * p.os + n;
    const E *plus = static_cast<const E *>(p.add) + m * p.as + n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = p.add && 16 * h + 2 * i < rows ? to_f(plus[(16 * h + 2 * i) * p.as]) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 16 * h + 2 * i;
            if (row < rows) to[row * p.os] = from_f<E>(own[(row + (lane >> 4)) * 17 + (lane & 15)] + a[i]);
        }
    }
}

template <typename E, int BN>
__global__ void __launch_bounds__(kPairThreads, 1) mm_pair_kernel(const __grid_constant__ MatmulArgs args, int wide) {
    using S = PairShape<BN>;
    constexpr bool kSums = sizeof(E) == 4;
    extern __shared__ unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char *scales = ring + S::kStage * S::kStages;
    unsigned char *staging = scales + S::kScaleStage * kScaleStages;   // 512-byte aligned
    __shared__ uint64_t full[S::kStages], empty[S::kStages], sfull[kScaleStages], sempty[kScaleStages], tfull[S::kBuffers], tempty[S::kBuffers];
    __shared__ uint32_t tmem_base;
    const MatmulParams &p = args.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int64_t down = ceil_div(p.a.rows, 2 * kRows), across = ceil_div(p.b.rows, BN), tiles = down * across;
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int blocks = (int)ceil_div(p.K, kFp8Block);
    const int segment = kSums ? kSegment : blocks;
    const int groups = (int)ceil_div(blocks, 4);                       // of scales per tile
    const int64_t all = pair < tiles ? ((tiles - pair - 1) / pairs + 1) * groups : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < kScaleStages; ++i) mbar_init(&sfull[i], rank == 0 ? 33 : 32), mbar_init(&sempty[i], 1);
        for (int i = 0; i < S::kBuffers; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 2 * kStoreWarps);
        fence_mbar_init();
    }
    if (warp == 3) tmem_alloc_pair(&tmem_base, S::kCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t acc = tmem_base, sf = acc + S::kBuffers * BN;
    bool ok = true;
    if (warp == 0) {
        // ---- tiles of both operands; the bytes of both CTAs count on the first one's barrier
        const bool issuer = elect_one();
        Slot<S::kStages> slot;
        int loads = 0;
        const uint32_t bars = mapa_shared(smem_u32(full), 0);
        for (int64_t t = pair; ok && t < tiles; t += pairs) {
            int64_t i, j;
            tile_at(t, down, across, i, j);
            const int ra = (int)(i * 2 * kRows + rank * kRows), rb = (int)(j * BN + rank * (BN / 2));
            for (int k = 0; k < blocks; ++k) {
                // (a wait for the turn before the first returns at once)
                if (!warp_wait<false>(&empty[slot.at], slot.turn ^ 1)) {
                    ok = false;
                    break;
                }
                unsigned char *at = ring + slot.at * S::kStage;
                if (issuer) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[slot.at], 2 * S::kStage);
                    tma_load_2d_pair(at, &args.a, bars + 8 * slot.at, k * kFp8Block, ra);
                    tma_load_2d_pair(at + kRows * kFp8Block, &args.b, bars + 8 * slot.at, k * kFp8Block, rb);
                }
                slot.next();
                loads = min(loads + 1, S::kStages);
            }
        }
        if (rank == 0)   // the copies end before the CTAs do
            for (int m = 0; m < loads; ++m) {
                slot.at = slot.at == 0 ? S::kStages - 1 : slot.at - 1;
                if (slot.at == S::kStages - 1) slot.turn ^= 1;
                if (!warp_wait<false>(&full[slot.at], slot.turn)) ok = false;
            }
    } else if (warp == 1 && rank == 0) {
        // ---- MMAs of the pair
        const bool issuer = elect_one();
        Slot<S::kStages> slot;
        Slot<kScaleStages> scale;
        Slot<S::kBuffers> sum;
        const uint64_t a0 = sdesc_sw128(smem_u32(ring), 16, 1024), s0 = sdesc_plain(smem_u32(scales), 128);
        const uint32_t idesc = idesc_mx8(2 * kRows, BN, p.a.dtype == kE5M2, p.b.dtype == kE5M2, 0);
        for (int64_t t = pair; ok && t < tiles; t += pairs) {
            for (int k0 = 0; ok && k0 < blocks; k0 += segment) {
                if (!warp_wait<false>(&tempty[sum.at], sum.turn ^ 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t to = acc + sum.at * BN;
                const int k1 = min(blocks, k0 + segment);
                bool ready = false;   // this lane has seen the next stage full
                for (int k = k0; k < k1; ++k) {
                    const uint32_t set = sf + (scale.at & 1) * S::kSet;
                    if (k % 4 == 0) {
                        if (!warp_wait<true>(&sfull[scale.at], scale.turn)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t from = s0 + scale.at * (S::kScaleStage >> 4);
                        if (issuer) {
#pragma unroll
                            for (int c = 0; c < S::kScaleStage / 512; ++c) tmem_copy_scales_pair(set + 4 * c, from + 32 * c);
                            mma_commit_pair(&sempty[scale.at]);
                        }
                    }
                    if (!__all_sync(0xffffffffu, ready) && !warp_wait<false>(&full[slot.at], slot.turn)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a0 + slot.at * (S::kStage >> 4), bd = ad + (kRows * kFp8Block >> 4);
                    const uint32_t id = idesc | (k & 3) << 4 | (uint32_t)(k & 3) << 29;
                    const int here = slot.at;
                    slot.next();
                    ready = mbar_try_wait(&full[slot.at], slot.turn);   // its answer is looked at after the MMAs' issue
                    if (issuer) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) mma_mx8_pair(to, ad + 2 * q, bd + 2 * q, id, set, set + 4, k != k0 || q > 0);
                        mma_commit_pair(&empty[here]);
                    }
                    if (k % 4 == 3 || k == blocks - 1) scale.next();
                }
                if (issuer) mma_commit_pair(&tfull[sum.at]);
                sum.next();
            }
        }
    } else if (warp == 1) {
        // ---- the second CTA's scales are there: told to the first by a warp that has no copies on
        // their way, because a release for the cluster waits for all of a thread's
        Slot<kScaleStages> scale;
        const uint32_t bars = mapa_shared(smem_u32(sfull), 0);
        for (int64_t n = 0; n < all; ++n) {
            ok = warp_wait<false>(&sfull[scale.at], scale.turn);
            if (!ok) break;
            if (lane == 0) mbar_arrive_remote(bars + 8 * scale.at);
            scale.next();
        }
    } else if (warp == 2) {
        // ---- scales: of this CTA's rows of a, and of all rows of b
        ScaleRows<kRows> rows_a;
        ScaleRows<BN> rows_b;
        int64_t t = pair;
        int g = 0;
        Slot<kScaleStages> in, out;
        for (int64_t n = 0; n < all + kAhead; ++n) {
            if (n < all) {
                if (g == 0) {
                    int64_t i, j;
                    tile_at(t, down, across, i, j);
                    rows_a.set(p.a, i * 2 * kRows + rank * kRows, lane);
                    rows_b.set(p.b, j * BN, lane);
                }
                ok = wait_for<false>(&sempty[in.at], in.turn ^ 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t at = smem_u32(scales + in.at * S::kScaleStage);
                const int bytes = min(4, blocks - 4 * g);
                rows_a.copy(at, bytes, lane);
                rows_b.copy(at + 512, bytes, lane);
                in.next();
                if (++g == groups) g = 0, t += pairs;
            }
            copies_commit();
            if (n >= kAhead) {
                copies_wait<kAhead>();
                fence_proxy_async_smem();
                mbar_arrive(&sfull[out.at]);
                out.next();
            }
        }
        copies_wait<0>();
    } else if (warp >= 4) {
        // ---- accumulators to out: lanes 32 (warp % 4) .. + 31, one half of the columns
        const int part = warp & 3, half = (warp - 4) >> 2;
        constexpr int kMost = (BN / 2 + 31) / 32 * 32;      // of the first half; the second may be shorter
        constexpr int V = 16 / sizeof(E);
        const int cols = half ? BN - kMost : kMost;
        unsigned char *own = staging + (warp - 4) * kStoreBuffer;
        Slot<S::kBuffers> sum;
        const uint32_t bars = mapa_shared(smem_u32(tempty), 0);
        for (int64_t t = pair; ok && t < tiles; t += pairs) {
            int64_t ti, tj;
            tile_at(t, down, across, ti, tj);
            const int64_t m0 = ti * 2 * kRows + rank * kRows + part * 32, n0 = tj * BN + half * kMost;
            const int64_t left = p.b.rows - n0;              // columns of out from here on
            const E *plus = p.add ? static_cast<const E *>(p.add) + (m0 + lane) * p.as + n0 : nullptr;
            const bool my_row = m0 + lane < p.a.rows;
            // this lane's row: fp32, or 16-bit values that begin as the addend's
            float f[kSums ? kMost : 1];
            Pack<E, V> o[kSums ? 1 : kMost / V];
            if constexpr (!kSums) {
                if (wide && plus) {
#pragma unroll
                    for (int c = 0; c < kMost; c += V)
                        if (c < cols) o[c / V] = ld_row<E, V>(plus + c, my_row ? (int)min(left - c, (int64_t)V) : 0);
                }
            }
            for (int k = 0; k < blocks; k += segment) {
                const int buf = sum.at;
                ok = warp_wait<false>(&tfull[buf], sum.turn);
                if (!ok) break;
                sum.next();
                tc_fence_after();
                const uint32_t from = tmem_addr(acc, part * 32, buf * BN + half * kMost);
                if constexpr (kSums) {
#pragma unroll
                    for (int c = 0; c < kMost; c += 32) {
                        if (c >= cols) break;
                        float r[32];
                        tmem_ld32(from + c, r);
                        tmem_ld_wait();
                        if (k == 0) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[c + e] = r[e];
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[c + e] += r[e];
                        }
                    }
                } else if (wide) {
#pragma unroll
                    for (int c = 0; c < kMost; c += 32) {
                        if (c >= cols) break;
                        float r[32];
                        tmem_ld32(from + c, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e += V) {
                            float (&v)[V] = reinterpret_cast<float (&)[V]>(r[e]);
                            if (plus) {
                                float a[V];
                                unpack<E, V>(o[(c + e) / V], a);
                                add_n<V>(v, v, a);
                            }
                            st_f<E, V>(o[(c + e) / V].e, v);
                        }
                    }
                } else {
                    // rows that no wide access fits: 16 columns at a time through shared memory
#pragma unroll 1
                    for (int c = 0; c < cols; c += 16) {
                        float r[16];
                        tmem_ld16(from + c, r);
                        tmem_ld_wait();
                        st_narrow<E>(p, r, reinterpret_cast<float *>(own), m0, n0 + c, lane);
                    }
                }
                tc_fence_before();
                if (lane == 0) mbar_arrive_remote(bars + 8 * buf);
            }
            if (!ok) break;
            if constexpr (kSums) {
                if (!wide) {
#pragma unroll
                    for (int c = 0; c < kMost; c += 16)
                        if (c < cols) st_narrow<E>(p, reinterpret_cast<float (&)[16]>(f[c]), reinterpret_cast<float *>(own), m0, n0 + c, lane);
                }
            }
            if (!wide || m0 >= p.a.rows) continue;
            // 64 bytes of every row to the buffer (16-byte piece j of row r at j ^ (r / 2 % 4), the
            // 64-byte swizzle), and from there by a tensor store, which leaves out what is outside
            constexpr int kStep = 64 / sizeof(E);
#pragma unroll
            for (int c = 0; c < kMost; c += kStep) {
                if (c >= cols || c >= left) break;
                if (lane == 0) bulk_wait_read0();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    Pack<E, V> piece;
                    if constexpr (kSums) {
                        float (&v)[V] = reinterpret_cast<float (&)[V]>(f[c + j * V]);
                        if (plus) {
                            float a[V];
                            unpack<E, V>(ld_row<E, V>(plus + c + j * V, my_row ? (int)min(left - c - j * V, (int64_t)V) : 0), a);
                            add_n<V>(v, v, a);
                        }
                        st_f<E, V>(piece.e, v);
                    } else {
                        piece = o[c / V + j];
                    }
                    *reinterpret_cast<Pack<E, V> *>(own + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) = piece;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&args.out, own, (int)(n0 + c), (int)m0);
                    bulk_commit();
                }
            }
        }
        if (lane == 0) bulk_wait0();
    }
    if (!ok && p.err) atomicExch(p.err, kErrTimeout);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // nothing of the pair is still to arrive at the other CTA
    if (warp == 3) tmem_dealloc_pair(acc, S::kCols);
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

// out for tensor stores of 64 bytes by 32 rows.
bool encode_out(CUtensorMap &map, const MatmulParams &p) {
    const auto encode = chunk::encode_fn();
    if (!encode) return false;
    const size_t e = dtype_bytes(p.dtype);
    const cuuint64_t dims[2] = {(cuuint64_t)p.b.rows, (cuuint64_t)p.a.rows}, strides[1] = {(cuuint64_t)p.os * e};
    const cuuint32_t box[2] = {(cuuint32_t)(64 / e), 32}, step[2] = {1, 1};
    const CUtensorMapDataType type = p.dtype == kBF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : p.dtype == kFP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    return encode(&map, type, 2, p.out, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

template <typename E, int BN>
cudaError_t run_pair(MatmulArgs &args, int sms, cudaStream_t stream) {
    using S = PairShape<BN>;
    constexpr auto kernel = mm_pair_kernel<E, BN>;
    cudaError_t e = allow_smem<kernel>(S::kSmem);
    if (e != cudaSuccess) return e;
    MatmulParams &p = args.p;
    if (!encode_operand(args.a, p.a, p.K, kRows) || !encode_operand(args.b, p.b, p.K, BN / 2)) return cudaErrorInvalidValue;
    constexpr int V = 16 / sizeof(E);
    const int wide = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.os % V == 0 &&
                     (!p.add || (reinterpret_cast<uintptr_t>(p.add) % 16 == 0 && p.as % V == 0));
    if (wide && !encode_out(args.out, p)) return cudaErrorInvalidValue;
    const int64_t tiles = ceil_div(p.a.rows, 2 * kRows) * ceil_div(p.b.rows, BN);
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(2 * (unsigned)std::min(tiles, (int64_t)sms / 2));
    c.blockDim = dim3(kPairThreads);
    c.dynamicSmemBytes = S::kSmem;
    c.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args, wide);
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
        if (p.a.rows > 256) {
            const char *bn = getenv("MM_BN");
            switch (bn ? atoi(bn) : 224) {
                case 128: return run_pair<E, 128>(args, sms, stream);
                case 192: return run_pair<E, 192>(args, sms, stream);
                case 256: return run_pair<E, 256>(args, sms, stream);
                default: return run_pair<E, 224>(args, sms, stream);
            }
        }
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
