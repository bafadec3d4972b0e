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
constexpr uint64_t kLate = kWait / 100;     // of copies under way where a wait has expired already
constexpr int kRows = 128;                  // rows of b per tile: the MMA's M, TMEM's lanes
constexpr int kScaleStages = 8, kAhead = 4;   // groups of 4 blocks' scales: places, and on their way
// Blocks of K in one accumulator where the output has 32 bits.  The tensor cores cut an accumulator at
// each MMA, always towards zero, so that over a long K that would cost more than fp32's own rounding;
// the sums of the segments are added in registers.
constexpr int kSegment = 64;

// Waits of the pipelines.  Reading the GPU's timer takes longer than a stage does, so it is read
// once in many tries only.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, uint64_t limit = kWait) {
    uint64_t t0 = 0;
    for (uint32_t tries = 0;; ++tries) {
        if (CLUSTER ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) return true;
        if (tries % 4096 == 4095) {
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
    __device__ __forceinline__ void set(const Fp8Operand &o, int64_t row0, int block, int lane) {   // from this block on
        in = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int64_t r = row0 + 32 * w + lane;
            const bool some = 32 * w + lane < N && r < o.rows;
            row[w] = o.s + (some ? (o.tile ? r / kFp8Block : r) * o.s_stride + block : 0);
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

// ---- few rows of a: one tile of 128 rows of b by BT rows of a per cluster of `split` CTAs, which
// share K and join their sums through distributed shared memory, each for a part of the rows of a.
// The rows of b, of which nearly all bytes are, lie along the MMA's M, so that tiles are full however
// few rows a has.  Two CTAs per SM keep up to 180 KB of loads in flight.
//
// Bound by reading b: 1 x 8192 x 8192 takes 14.5 us, 16 rows 15.9, 64 rows 17.6 (64 x 8192 x 65536 90
// us), and 67 MB more of b 10.7 us more (6.3 TB/s); 3.5 us go to the way into the pipeline and out of
// it.  With one lane of a warp issuing behind a branch 1 x 8192 x 8192 took 21 us, with one CTA per SM
// 24 us, with the sums of one row at a time on their way 64 rows took 19.7 us.
//
// A long K has an accumulator for each segment, `sums` of them, which are added in registers at the
// end.  A CTA takes up to half of the SM's TMEM, so that the two of an SM never wait for each other's:
// CTAs of two clusters that did could wait in a circle.
template <int BT>
struct TileShape {
    static constexpr int kStage = (kRows + BT) * kFp8Block;
    static constexpr int kScaleStage = 1024;
    static constexpr int kStages = (113 * 1024 - 2048 - kScaleStage * kScaleStages) / kStage;
    static constexpr int kSmem = 1024 + kStage * kStages + kScaleStage * kScaleStages;
    static_assert(BT * kRows * 4 <= kStage * kStages, "the sums fit the ring");
    static constexpr int kSet = 8;                     // TMEM columns of scales
    static constexpr int kMostSums = (256 - 2 * kSet) / BT;
    static int cols(int sums) {                        // TMEM columns, a power of two
        int n = 32;
        while (n < sums * BT + 2 * kSet) n *= 2;
        return n;
    }
};

template <typename E, int BT>
__global__ void __launch_bounds__(128) mm_tile_kernel(const __grid_constant__ MatmulArgs args, int split, int segment, int sums, int cols) {
    using S = TileShape<BT>;
    extern __shared__ unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char *scales = ring + S::kStage * S::kStages;
    __shared__ uint64_t full[S::kStages], empty[S::kStages], sfull[kScaleStages], sempty[kScaleStages], done;
    __shared__ uint32_t tmem_base;
    const MatmulParams &p = args.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = blockIdx.x % split;
    const uint32_t tile = blockIdx.x / split, across = (uint32_t)ceil_div(p.b.rows, kRows);
    const int64_t m0 = (int64_t)(tile / across) * BT, n0 = (int64_t)(tile % across) * kRows;
    const int blocks = (int)ceil_div(p.K, kFp8Block);
    const int each = blocks / split, more = blocks - each * split;
    const int k0 = each * rank + min(rank, more), k1 = k0 + each + (rank < more);
    const int early = min(k1 - k0, S::kStages);        // loads that wait for nothing
    bool ok = true, issuer = false;
    const auto load = [&](int k, int at) {
        unsigned char *to = ring + at * S::kStage;
        mbar_arrive_expect_tx(&full[at], S::kStage);
        tma_box(to, args.b, &full[at], k * kFp8Block, (int)n0);
        tma_box(to + kRows * kFp8Block, args.a, &full[at], k * kFp8Block, (int)m0);
    };
    if (warp == 0) {
        issuer = elect_one();
        if (issuer) {
            for (int i = 0; i < S::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
            for (int i = 0; i < kScaleStages; ++i) mbar_init(&sfull[i], 32), mbar_init(&sempty[i], 1);
            mbar_init(&done, 1);
            fence_mbar_init();
        }
    } else if (warp == 1) {
        issuer = elect_one();
        tmem_alloc(&tmem_base, cols);
        tmem_relinquish();
    }
    wait_for_prior_kernels();
    allow_next_kernel();
    if (warp == 0 && issuer)
        for (int i = 0; i < early; ++i) load(k0 + i, i);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t acc = tmem_base, sf = acc + sums * BT;
    if (warp == 0) {
        Slot<S::kStages> slot;
        for (int k = k0 + early; k < k1; ++k) {
            ok = warp_wait<false>(&empty[slot.at], slot.turn);
            if (!ok) break;
            if (issuer) load(k, slot.at);
            slot.next();
        }
        // the copies end before the CTA does: the last loads of all slots, in order
        if (early < S::kStages) slot.at = 0;
        for (int i = 0; i < early; ++i) {
            if (!warp_wait<false>(&full[slot.at], early < S::kStages ? 0 : slot.turn, ok ? kWait : kLate)) ok = false;
            slot.next();
        }
    } else if (warp == 1) {
        Slot<S::kStages> slot;
        Slot<kScaleStages> scale;
        const uint64_t b0 = sdesc_sw128(smem_u32(ring), 16, 1024), s0 = sdesc_plain(smem_u32(scales), 128);
        const uint32_t idesc = idesc_mx8(kRows, BT, p.b.dtype == kE5M2, p.a.dtype == kE5M2, 0);
        uint32_t to = acc;
        for (int k = k0, in = 0; k < k1; ++k, ++in) {
            const uint32_t set = sf + (scale.at & 1) * S::kSet;
            if (in == segment) in = 0, to += BT;
            if (k % 4 == 0 || k == k0) {
                ok = warp_wait<false>(&sfull[scale.at], scale.turn);
                if (!ok) break;
                tc_fence_after();
                const uint64_t from = s0 + scale.at * (S::kScaleStage >> 4);
                if (issuer) {
                    tmem_copy_scales(set, from);
                    tmem_copy_scales(set + 4, from + 32);
                    mma_commit(&sempty[scale.at]);
                }
            }
            ok = warp_wait<false>(&full[slot.at], slot.turn);
            if (!ok) break;
            tc_fence_after();
            const uint64_t bd = b0 + slot.at * (S::kStage >> 4), ad = bd + (kRows * kFp8Block >> 4);
            const uint32_t id = idesc | (k & 3) << 4 | (uint32_t)(k & 3) << 29;
            if (issuer) {
#pragma unroll
                for (int q = 0; q < 4; ++q) mma_mx8(to, bd + 2 * q, ad + 2 * q, id, set, set + 4, in > 0 || q > 0);
                mma_commit(&empty[slot.at]);
            }
            slot.next();
            if (k % 4 == 3) scale.next();
        }
        if (issuer) mma_commit(&done);
    } else if (warp == 2) {
        // kAhead groups on their way while the ones before are handed over
        const int g0 = k0 / 4, groups = (k1 - 1) / 4 - g0 + 1;
        ScaleRows<kRows> rows_b;
        ScaleRows<BT> rows_a;
        rows_b.set(p.b, n0, 4 * g0, lane);
        rows_a.set(p.a, m0, 4 * g0, lane);
        Slot<kScaleStages> in, out;
        for (int i = 0; i < groups + kAhead; ++i) {
            if (i < groups) {
                ok = warp_wait<false>(&sempty[in.at], in.turn ^ 1);
                if (!ok) break;
                const uint32_t at = smem_u32(scales + in.at * S::kScaleStage);
                const int bytes = min(4, blocks - 4 * (g0 + i));
                rows_b.copy(at, bytes, lane);
                rows_a.copy(at + 512, bytes, lane);
                in.next();
            }
            copies_commit();
            if (i >= kAhead) {
                copies_wait<kAhead>();
                fence_proxy_async_smem();
                mbar_arrive(&sfull[out.at]);
                out.next();
            }
        }
        copies_wait<0>();
    }
    __syncwarp();
    if (!wait_for<false>(&done, 0, 2 * kWait)) ok = false;
    if (!ok && p.err) atomicExch(p.err, kErrTimeout);
    __syncwarp();
    tc_fence_after();
    const int64_t n = n0 + threadIdx.x;
    E *to = static_cast<E *>(p.out) + m0 * p.os + n;
    const E *plus = p.add ? static_cast<const E *>(p.add) + m0 * p.as + n : nullptr;
    const int real = (int)min(p.a.rows - m0, (int64_t)BT), here = n < p.b.rows ? real : 0;   // rows of a: all, and those to store
    // 16 rows' sums of all of this CTA's segments, in the order of K
    const auto summed = [&](int c, float (&r)[16]) {
        tmem_ld16(tmem_addr(acc, warp * 32, c), r);
        tmem_ld_wait();
        for (int k = k0 + segment, at = c + BT; k < k1; k += segment, at += BT) {
            float more[16];
            tmem_ld16(tmem_addr(acc, warp * 32, at), more);
            tmem_ld_wait();
            add_n<16>(r, r, more);
        }
    };
    if (split > 1) {
        // the ring is free: every load and MMA has ended
        float *parts = reinterpret_cast<float *>(ring) + threadIdx.x;   // [BT][128]
        for (int c = 0; c < real; c += 16) {
            float r[16];
            summed(c, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) parts[(c + j) * kRows] = r[j];
        }
        cluster_sync();
        const int rows = BT / split, c1 = min(rows * (rank + 1), real);
        const uint32_t mine = smem_u32(parts);
        for (int c = rows * rank; c < c1; c += 4) {      // 4 rows' sums on their way
            float v[4][8], add[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = min(c + i, c1 - 1);
                add[i] = plus && row < here ? to_f(plus[row * p.as]) : 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < split) v[i][q] = ld_cluster(mapa_shared(mine + row * kRows * 4, q));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float t = v[i][0];
#pragma unroll
                for (int q = 1; q < 8; ++q)
                    if (q < split) t += v[i][q];
                if (c + i < min(c1, here)) to[(c + i) * p.os] = from_f<E>(plus ? t + add[i] : t);
            }
        }
    } else {
        for (int c = 0; c < BT; c += 16) {
            float r[16], add[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) add[j] = plus && c + j < here ? to_f(plus[(c + j) * p.as]) : 0.f;
            summed(c, r);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < here) to[(c + j) * p.os] = from_f<E>(plus ? r[j] + add[j] : r[j]);
        }
    }
    tc_fence_before();
    if (split > 1) cluster_sync();   // the others have read this CTA's sums
    else __syncthreads();
    if (warp == 1) tmem_dealloc(acc, cols);
}

// ---- tiles of 256 rows of a by BN rows of b, each of a pair of CTAs.
//
// Each CTA of a pair loads its 128 rows of a and half of the rows of b, one thread of the first CTA
// issues the MMAs of both (cta_group::2), which halves what shared memory has to deliver for b.
// Warp 0 loads tiles, warp 2 scales, warp 1 issues, warps 4 to 11 empty the accumulators.
//   SPLIT = 1: pairs are persistent and walk the tiles, with two accumulators in TMEM, so that a
// tile's MMAs run while the one before is stored.  fp32 outputs take K in segments whose sums are
// added in registers.
//   SPLIT = 2, 4: few tiles; a cluster of SPLIT pairs shares a tile's K and joins the sums through
// distributed shared memory, each pair for its part of the columns.
//
// 8192 x 8192 x 8192 e4m3 to bf16: 363 to 374 us, 3.0 PFLOP/s, where calls follow one another for a
// second, under the power cap, and 302 us, 3.64 PFLOP/s, in short runs: 1.8 and 1.9 times what bf16
// products of a library reach on the same card; the tensor pipe is active for 83% of the time.  A weight
// gradient, 8192 x 2048 x 16384 to fp32 with an addend, 234 us and 212 (2.35 and 2.6 PFLOP/s).  A block
// of 128 of K costs an SM 256 + BN cycles to load at 64 bytes a cycle, and 2 BN to multiply: wide tiles
// for many, and where tiles are few more of them.
// What it took: all of a warp at the waits, one elected lane at the issue (4096^3 74 us instead of
// 80), scales in 8 groups of places with 4 on their way and handed to the other CTA by a warp that has
// no copies under way (8192^3 453 us, then 384, then 326), polling instead of suspended waits (512 x
// 2048 x 512 11.3 us, then 7.3), the accumulator's stores behind its return to the MMAs.
constexpr int kPairThreads = 384, kStoreWarps = 8;

// A store warp's buffers: two of 32 rows of 64 bytes for tensor stores, or one of 32 x 17 fp32.
constexpr int kStoreBuffer = 4096;

template <int BN, int SPLIT>
struct PairShape {
    static constexpr int kStage = (kRows + BN / 2) * kFp8Block;
    static constexpr int kScaleB = BN <= 128 ? 512 : 1024;
    static constexpr int kScaleStage = 512 + kScaleB;
    static constexpr int kStaging = kStoreWarps * kStoreBuffer;
    static constexpr int kStages = (227 * 1024 - 2048 - kStaging - kScaleStage * kScaleStages) / kStage;
    static constexpr int kSmem = 1024 + kStage * kStages + kScaleStage * kScaleStages + kStaging;
    static constexpr int kSet = 4 + kScaleB / 128;
    static constexpr int kBuffers = SPLIT > 1 ? 1 : 2, kCols = 512;
    static constexpr int kMost = (BN / 2 + 31) / 32 * 32;   // columns of a store warp, at most
    static constexpr int kSlice = kMost / SPLIT;            // SPLIT > 1: those that a pair finishes
    static_assert(kSmem <= 227 * 1024 && BN % 32 == 0 && kBuffers * BN + 2 * kSet <= kCols, "fits an SM");
    static_assert(SPLIT == 1 || (BN % 64 == 0 && kSlice % 16 == 0 && (SPLIT - 1) * kStoreWarps * kSlice * 128 <= kStage * kStages),
                  "the other pairs' sums fit the ring");
};

// Tile t of a grid of `down` x `across`: 8 tiles down, then across, so that the tiles in flight
// share rows of both operands in L2.
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t down, uint32_t across, uint32_t &i, uint32_t &j) {
    const uint32_t band = t / (8 * across), first = band * 8, high = min(down - first, 8u), in = t - band * 8 * across;
    j = in / high;
    i = first + in - j * high;
}

// 32 bytes in one load.
template <typename P>
__device__ __forceinline__ void ld_sector(const void *at, P (&to)[2]) {
    uint32_t u[8];
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "l"(at)
                 : "memory");
    static_assert(sizeof(to) == sizeof(u), "two groups of 16 bytes");
    memcpy(&to, u, sizeof(u));
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

// One element, where there is one (a branch around each of many would cost more than the access).
template <typename E>
__device__ __forceinline__ E ld_one(const E *at, bool there) {
    if constexpr (sizeof(E) == 4) {
        float v;
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t@q ld.global.f32 %0, [%1];\n\t}"
                     : "=f"(v) : "l"(at), "r"((int)there) : "memory");
        return v;
    } else {
        uint16_t v;
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b16 %0, 0;\n\t@q ld.global.b16 %0, [%1];\n\t}"
                     : "=h"(v) : "l"(at), "r"((int)there) : "memory");
        return *reinterpret_cast<E *>(&v);
    }
}
template <typename E>
__device__ __forceinline__ void st_one(E *at, E v, bool there) {
    if constexpr (sizeof(E) == 4)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q st.global.f32 [%0], %1;\n\t}" ::"l"(at), "f"(v), "r"((int)there) : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q st.global.b16 [%0], %1;\n\t}" ::"l"(at),
                     "h"(*reinterpret_cast<const uint16_t *>(&v)), "r"((int)there)
                     : "memory");
}

// out and its addend by single elements, 16 columns of 32 rows at a time: a lane takes column
// lane % 16 of every other row, so that neighbours take neighbours.
template <typename E>
struct NarrowRows {
    E *out;
    const E *add;
    int64_t os, as;   // two rows on
    int rows, cols;   // from this lane's first row and column on
    __device__ __forceinline__ NarrowRows(const MatmulParams &p, int64_t m0, int64_t n0, int lane) {
        const int64_t m = m0 + (lane >> 4), n = n0 + (lane & 15);
        out = static_cast<E *>(p.out) + m * p.os + n;
        add = p.add ? static_cast<const E *>(p.add) + m * p.as + n : nullptr;
        os = 2 * p.os, as = 2 * p.as;
        rows = (int)min(max(p.a.rows - m, (int64_t)0), (int64_t)32);
        cols = (int)min(p.b.rows - n, (int64_t)1 << 30);
    }
    // Column c of rows 0, 2, ..., 30 from this lane's first on (0 where there is no addend).
    __device__ __forceinline__ void addend(int c, E (&to)[16]) const {
        const E *at = add + c;
        const int some = add && c < cols ? rows : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i, at += as) to[i] = ld_one(at, 2 * i < some);
    }
    __device__ __forceinline__ void put(int c, const E (&v)[16]) const {
        E *at = out + c;
        const int some = c < cols ? rows : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i, at += os) st_one(at, v[i], 2 * i < some);
    }
    // From 16 columns of a row to a lane to this order.  `own`: 32 x 17 fp32 of shared memory.
    static __device__ __forceinline__ void turn(float *own, float *r, int lane) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 16; ++e) own[lane * 17 + e] = r[e];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = own[(2 * i + (lane >> 4)) * 17 + (lane & 15)];
    }
};

template <typename E, int BN, int SPLIT>
__global__ void __launch_bounds__(kPairThreads, 1) mm_pair_kernel(const __grid_constant__ MatmulArgs args, int wide) {
    using S = PairShape<BN, SPLIT>;
    constexpr bool kSums = sizeof(E) == 4 && SPLIT == 1;
    extern __shared__ unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char *scales = ring + S::kStage * S::kStages;
    unsigned char *staging = scales + S::kScaleStage * kScaleStages;   // 512-byte aligned
    __shared__ uint64_t full[S::kStages], empty[S::kStages], sfull[kScaleStages], sempty[kScaleStages], tfull[S::kBuffers], tempty[S::kBuffers];
    __shared__ uint32_t tmem_base;
    const MatmulParams &p = args.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // this CTA's place in its pair, the pair's first CTA in the cluster, both as a mask
    const uint32_t in_cluster = cluster_ctarank(), rank = in_cluster & 1, first = in_cluster & ~1u;
    const uint16_t both_ctas = (uint16_t)(3u << first);
    const int part = SPLIT > 1 ? first >> 1 : 0;
    const uint32_t down = (uint32_t)ceil_div(p.a.rows, 2 * kRows), across = (uint32_t)ceil_div(p.b.rows, BN), tiles = down * across;
    const uint32_t pair = blockIdx.x / (2 * SPLIT), pairs = gridDim.x / (2 * SPLIT);
    // blocks of K: all, or this pair's part, which begins at a group of 4
    const int blocks = (int)ceil_div(p.K, kFp8Block), groups = (blocks + 3) / 4, each = groups / SPLIT, over = groups - each * SPLIT;
    const int k_begin = SPLIT > 1 ? 4 * (each * part + min(part, over)) : 0;
    const int k_end = SPLIT > 1 ? min(k_begin + 4 * (each + (part < over)), blocks) : blocks;
    const int segment = kSums ? kSegment : blocks;
    const bool narrow_rows = __builtin_expect(wide == 0, 0);   // their code off the others' way
    if (threadIdx.x == 0) {
        prefetch_map(&args.a);
        prefetch_map(&args.b);
        for (int i = 0; i < S::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < kScaleStages; ++i) mbar_init(&sfull[i], rank == 0 ? 33 : 32), mbar_init(&sempty[i], 1);
        for (int i = 0; i < S::kBuffers; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 2 * kStoreWarps);
        fence_mbar_init();
    }
    if (warp == 3) tmem_alloc_pair(&tmem_base, S::kCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    wait_for_prior_kernels();
    allow_next_kernel();
    tc_fence_after();
    const uint32_t acc = tmem_base, sf = acc + S::kBuffers * BN;
    bool ok = true;
    if (warp == 0) {
        // ---- tiles of both operands; the bytes of both CTAs count on the first one's barrier
        const bool issuer = elect_one();
        Slot<S::kStages> slot;
        int loads = 0;
        const uint32_t bars = mapa_shared(smem_u32(full), first);
        for (uint32_t t = pair; ok && t < tiles; t += pairs) {
            uint32_t ti, tj;
            tile_at(t, down, across, ti, tj);
            const int ra = (int)(ti * (2 * kRows) + rank * kRows), rb = (int)(tj * BN + rank * (BN / 2));
            for (int k = k_begin; k < k_end; ++k) {
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
                if (!warp_wait<false>(&full[slot.at], slot.turn, ok ? kWait : kLate)) ok = false;
            }
    } else if (warp == 1 && rank == 0) {
        // ---- MMAs of the pair
        const bool issuer = elect_one();
        Slot<S::kStages> slot;
        Slot<kScaleStages> scale;
        Slot<S::kBuffers> sum;
        const uint64_t a0 = sdesc_sw128(smem_u32(ring), 16, 1024), s0 = sdesc_plain(smem_u32(scales), 128);
        const uint32_t idesc = idesc_mx8(2 * kRows, BN, p.a.dtype == kE5M2, p.b.dtype == kE5M2, 0);
        for (uint32_t t = pair; ok && t < tiles; t += pairs) {
            uint32_t ti, tj;
            tile_at(t, down, across, ti, tj);
            for (int k0 = k_begin; ok && k0 < k_end; k0 += segment) {
                if (!warp_wait<false>(&tempty[sum.at], sum.turn ^ 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t to = acc + sum.at * BN;
                const int k1 = min(k_end, k0 + segment);
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
                            mma_commit_pair(&sempty[scale.at], both_ctas);
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
                    ready = mbar_test_wait(&full[slot.at], slot.turn);   // its answer is looked at after the MMAs' issue
                    if (issuer) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) mma_mx8_pair(to, ad + 2 * q, bd + 2 * q, id, set, set + 4, k != k0 || q > 0);
                        mma_commit_pair(&empty[here], both_ctas);
                    }
                    if (k % 4 == 3 || k == blocks - 1) scale.next();
                }
                if (issuer) mma_commit_pair(&tfull[sum.at], both_ctas);
                sum.next();
            }
        }
    } else if (warp == 1) {
        // ---- the second CTA's scales are there: told to the first by a warp that has no copies on
        // their way, because a release for the cluster waits for all of a thread's
        Slot<kScaleStages> scale;
        const uint32_t bars = mapa_shared(smem_u32(sfull), first);
        for (uint32_t t = pair; ok && t < tiles; t += pairs) {
            uint32_t ti, tj;
            tile_at(t, down, across, ti, tj);
            for (int k = k_begin; k < k_end; k += 4) {
                ok = warp_wait<false>(&sfull[scale.at], scale.turn);
                if (!ok) break;
                if (lane == 0) mbar_arrive_remote(bars + 8 * scale.at);
                scale.next();
            }
        }
    } else if (warp == 2) {
        // ---- scales: of this CTA's rows of a, and of all rows of b; kAhead groups of 4 blocks are on
        // their way while the ones before are handed over
        ScaleRows<kRows> rows_a;
        ScaleRows<BN> rows_b;
        Slot<kScaleStages> in, out;
        int waiting = 0;                                  // groups on their way
        const auto hand_over = [&]() {
            fence_proxy_async_smem();
            mbar_arrive(&sfull[out.at]);
            out.next();
            --waiting;
        };
        for (uint32_t t = pair; ok && t < tiles; t += pairs) {
            uint32_t ti, tj;
            tile_at(t, down, across, ti, tj);
            rows_a.set(p.a, (int64_t)ti * (2 * kRows) + rank * kRows, k_begin, lane);
            rows_b.set(p.b, (int64_t)tj * BN, k_begin, lane);
            for (int k = k_begin; k < k_end; k += 4) {
                ok = warp_wait<false>(&sempty[in.at], in.turn ^ 1);
                if (!ok) break;
                const uint32_t at = smem_u32(scales + in.at * S::kScaleStage);
                const int bytes = min(4, blocks - k);
                rows_a.copy(at, bytes, lane);
                rows_b.copy(at + 512, bytes, lane);
                in.next();
                copies_commit();
                if (++waiting > kAhead) {
                    copies_wait<kAhead>();
                    hand_over();
                }
            }
        }
        copies_wait<0>();
        while (ok && waiting > 0) hand_over();
    } else if (warp >= 4) {
        if constexpr (SPLIT > 1) {
            ok = warp_wait<false>(&tfull[0], 0);
            tc_fence_after();
        } else {
            // ---- accumulators to out: lanes 32 (warp % 4) .. + 31, one half of the columns
            const int quarter = warp & 3, half = (warp - 4) >> 2;
            constexpr int kMost = S::kMost;              // of the first half; the second may be shorter
            constexpr int V = 16 / sizeof(E), kStep = 64 / sizeof(E);   // elements of 16 bytes, and of 64
            const int cols = half ? BN - kMost : kMost;
            unsigned char *own = staging + (warp - 4) * kStoreBuffer;
            uint32_t turn = 0;                           // of the two store buffers, over all tiles
            Slot<S::kBuffers> sum;
            const uint32_t bars = mapa_shared(smem_u32(tempty), first);
            for (uint32_t t = pair; ok && t < tiles; t += pairs) {
                uint32_t ti, tj;
                tile_at(t, down, across, ti, tj);
                const int64_t m0 = (int64_t)ti * (2 * kRows) + rank * kRows + quarter * 32, n0 = (int64_t)tj * BN + half * kMost;
                const int64_t left = p.b.rows - n0;          // columns of out from here on
                const E *plus = p.add ? static_cast<const E *>(p.add) + (m0 + lane) * p.as + n0 : nullptr;
                const bool my_row = m0 + lane < p.a.rows;
                // a sector at a time where rows start with one
                const auto addend = [&](int c, Pack<E, V> (&to)[2]) {
                    const int n = my_row ? (int)min(left - c, (int64_t)(2 * V)) : 0;
                    if (kSums && wide == 2 && n >= 2 * V) {
                        ld_sector(plus + c, to);
                    } else {
                        to[0] = ld_row<E, V>(plus + c, n);
                        to[1] = ld_row<E, V>(plus + c + V, n - V);
                    }
                };
                // 64 bytes of every row to one of the two buffers (16-byte piece j of row r at
                // j ^ (r / 2 % 4), the 64-byte swizzle), and from there by a tensor store, which leaves
                // out rows that are outside and what is outside of a row but for the rest of the last 16
                // bytes: a row that ends inside of those is stored by single elements.  The buffers alternate with the stores, also from a tile to the
                // next, which may have an odd number: the one store that the wait leaves out is always the
                // other buffer's.
                const auto send = [&](int c, const Pack<E, V> (&piece)[4]) {
                    if (c >= left || m0 >= p.a.rows) return;
                    unsigned char *buffer = own + turn * 2048;
                    if (lane == 0) bulk_wait_read1();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) *reinterpret_cast<Pack<E, V> *>(buffer + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) = piece[j];
                    if (left - c < kStep && (left - c) % V) {
                        __syncwarp();
                        E *to = static_cast<E *>(p.out) + m0 * p.os + n0 + c + lane;
#pragma unroll 1
                        for (int r = 0; r < 32; ++r, to += p.os)
                            if (lane < left - c && m0 + r < p.a.rows)
                                *to = reinterpret_cast<const E *>(buffer + r * 64 + ((lane / V ^ (r >> 1 & 3)) << 4))[lane % V];
                        __syncwarp();
                        return;                              // (no store reads this buffer: it is the next one's, too)
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&args.out, buffer, (int)(n0 + c), (int)m0);
                        bulk_commit();
                    }
                    turn ^= 1;
                };
                // this lane's row (or where rows are not wide: its share of 32 rows), which begins as the
                // addend's, read while the MMAs run; the sums of the segments of K are added to it
                Pack<E, V> o[kMost / V];
                E (&single)[kMost] = reinterpret_cast<E (&)[kMost]>(o);
                if (narrow_rows) {
                    const NarrowRows<E> narrow(p, m0, n0, lane);
#pragma unroll
                    for (int c = 0; c < kMost; c += 16)
                        if (c < cols) narrow.addend(c, reinterpret_cast<E (&)[16]>(single[c]));
                } else if (plus) {
#pragma unroll
                    for (int c = 0; c < kMost; c += 2 * V)
                        if (c < cols) addend(c, reinterpret_cast<Pack<E, V> (&)[2]>(o[c / V]));
                } else if (kSums) {
#pragma unroll
                    for (int c = 0; c < kMost; ++c) single[c] = from_f<E>(0.f);
                }
                int k = 0;
                do {
                    const int buf = sum.at;
                    ok = warp_wait<false>(&tfull[buf], sum.turn);
                    if (!ok) break;
                    sum.next();
                    tc_fence_after();
                    const uint32_t from = tmem_addr(acc, quarter * 32, buf * BN + half * kMost);
                    // this lane's kStep columns from c on, added to what is held of them
                    const auto join = [&](int c, float (&r)[kStep]) {
#pragma unroll
                        for (int e = 0; e < kStep; e += V) {
                            float (&v)[V] = reinterpret_cast<float (&)[V]>(r[e]);
                            if (kSums || plus) {
                                float a[V];
                                unpack<E, V>(o[(c + e) / V], a);
                                add_n<V>(v, v, a);
                            }
                            st_f<E, V>(o[(c + e) / V].e, v);
                        }
                    };
                    const auto sums_at = [&](int c, float (&r)[kStep]) {
                        if constexpr (kStep == 32) tmem_ld32(from + c, r);
                        else tmem_ld16(from + c, r);
                        tmem_ld_wait();
                    };
                    if (!narrow_rows) {
#pragma unroll
                        for (int c = 0; c < kMost; c += kStep) {
                            if (c >= cols) break;
                            float r[kStep];
                            sums_at(c, r);
                            join(c, r);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < kMost; c += kStep) {
                            if (c >= cols) break;
                            float r[kStep];
                            sums_at(c, r);
#pragma unroll
                            for (int e = 0; e < kStep; e += 16) NarrowRows<E>::turn(reinterpret_cast<float *>(own), r + e, lane);
                            join(c, r);
                        }
                    }
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_remote_only(bars + 8 * buf);
                } while (kSums && (k += segment) < blocks);
                if (!ok) break;
                if (!narrow_rows) {
#pragma unroll
                    for (int c = 0; c < kMost; c += kStep)
                        if (c < cols) send(c, reinterpret_cast<const Pack<E, V> (&)[4]>(o[c / V]));
                } else {
                    const NarrowRows<E> narrow(p, m0, n0, lane);
#pragma unroll
                    for (int c = 0; c < kMost; c += 16)
                        if (c < cols) narrow.put(c, reinterpret_cast<const E (&)[16]>(single[c]));
                }
            }
            if (lane == 0) bulk_wait0();
        }
    }
    if constexpr (SPLIT > 1) {
        // Each store warp sends the sums of the other pairs' columns to the same warp of their CTAs,
        // into the ring, which is free once every MMA of the cluster has ended, and adds up its own
        // columns in the order of K.
        __syncwarp();
        tc_fence_before();
        cluster_sync();
        tc_fence_after();
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        constexpr int kSlice = S::kSlice;
        const uint32_t from = tmem_addr(acc, quarter * 32, half * S::kMost);
        float *box = reinterpret_cast<float *>(ring) + (warp - 4) * (SPLIT - 1) * kSlice * 32 + lane;
        if (warp >= 4 && ok) {
#pragma unroll 1
            for (int q = 0; q < SPLIT; ++q) {
                if (q == part) continue;
                const uint32_t to = mapa_shared(smem_u32(box + (part < q ? part : part - 1) * kSlice * 32), 2 * q + rank);
#pragma unroll
                for (int c = 0; c < kSlice; c += 16) {
                    float r[16];
                    tmem_ld16(from + q * kSlice + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) st_cluster(to + (c + e) * 128, r[e]);
                }
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= 4 && ok) {
            uint32_t ti, tj;
            tile_at(pair, down, across, ti, tj);
            constexpr int V = 16 / sizeof(E);
            const int64_t m0 = (int64_t)ti * (2 * kRows) + rank * kRows + quarter * 32;
            const int64_t n0 = (int64_t)tj * BN + half * S::kMost + part * kSlice, left = p.b.rows - n0;
            const bool my_row = m0 + lane < p.a.rows;
            E *to = static_cast<E *>(p.out) + (m0 + lane) * p.os + n0;
            const E *plus = p.add ? static_cast<const E *>(p.add) + (m0 + lane) * p.as + n0 : nullptr;
            // 16 columns' sums of all parts
            const auto joined = [&](int c, float (&s)[16]) {
                float r[16];
                tmem_ld16(from + part * kSlice + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = part == 0 ? r[e] : box[(c + e) * 32];
#pragma unroll
                for (int q = 1; q < SPLIT; ++q)
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] += q == part ? r[e] : box[((q < part ? q : q - 1) * kSlice + c + e) * 32];
            };
            if (narrow_rows) {
                const NarrowRows<E> narrow(p, m0, n0, lane);
                E next[16];
                narrow.addend(0, next);
#pragma unroll 1
                for (int c = 0; c < kSlice; c += 16) {
                    float s[16];
                    E v[16];
                    joined(c, s);
                    NarrowRows<E>::turn(reinterpret_cast<float *>(staging + (warp - 4) * kStoreBuffer), s, lane);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = from_f<E>(plus ? s[e] + to_f(next[e]) : s[e]);
                    if (c + 16 < kSlice) narrow.addend(c + 16, next);
                    narrow.put(c, v);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < kSlice; c += 16) {
                    float s[16];
                    Pack<E, V> a[16 / V];
                    if (plus) {
#pragma unroll
                        for (int e = 0; e < 16; e += V) a[e / V] = ld_row<E, V>(plus + c + e, my_row ? (int)min(left - c - e, (int64_t)V) : 0);
                    }
                    joined(c, s);
#pragma unroll
                    for (int e = 0; e < 16; e += V) {
                        float (&v)[V] = reinterpret_cast<float (&)[V]>(s[e]);
                        if (plus) {
                            float b[V];
                            unpack<E, V>(a[e / V], b);
                            add_n<V>(v, v, b);
                        }
                        if (!my_row) continue;
                        if (left - c - e >= V) {
                            st_f<E, V>(to + c + e, v);
                        } else {
#pragma unroll
                            for (int x = 0; x < V; ++x)
                                if (x < left - c - e) to[c + e + x] = from_f<E>(v[x]);
                        }
                    }
                }
            }
        }
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
cudaError_t launch_tile(MatmulArgs &args, int sms, cudaStream_t stream) {
    using S = TileShape<BT>;
    constexpr auto kernel = mm_tile_kernel<E, BT>;
    const cudaError_t e = allow_smem<kernel>(S::kSmem);
    if (e != cudaSuccess) return e;
    const MatmulParams &p = args.p;
    if (!encode_operand(args.a, p.a, p.K, BT) || !encode_operand(args.b, p.b, p.K, kRows)) return cudaErrorInvalidValue;
    // as many parts of K as two CTAs per SM hold, of 4 blocks or more; for 32-bit outputs also as many
    // as leave a part kSegment blocks
    const int64_t tiles = ceil_div(p.b.rows, kRows) * ceil_div(p.a.rows, BT), blocks = ceil_div(p.K, kFp8Block);
    int split = 1;
    while (split < 8 && ((tiles * split * 2 <= 2 * sms && blocks >= 8 * split) || (p.dtype == kFP32 && blocks > split * kSegment))) split *= 2;
    // longer segments only of 16-bit outputs (run_tile)
    const int64_t each = ceil_div(blocks, split), segment = std::max((int64_t)kSegment, ceil_div(each, S::kMostSums));
    const int sums = (int)ceil_div(each, segment);
    return launch_early(kernel, tiles * split, dim3(128), S::kSmem, stream, split, args, split, (int)segment, sums, S::cols(sums));
}

// A 32-bit output of a K with more segments than 8 CTAs have accumulators for takes it a piece at a time,
// each added to what the ones before have left in out.  (40 x 256 x 262144 with an addend 94 us; by pairs
// of CTAs, which empty their accumulators after each segment, 508 us.)
template <typename E, int BT>
cudaError_t run_tile(MatmulArgs &args, int sms, cudaStream_t stream) {
    const MatmulParams whole = args.p;
    const int64_t most = whole.dtype == kFP32 ? int64_t(8) * TileShape<BT>::kMostSums * kSegment * kFp8Block : whole.K;
    MatmulParams &p = args.p;
    for (int64_t k = 0; k < whole.K; k += most) {
        p.K = std::min(most, whole.K - k);
        p.a.q = static_cast<const uint8_t *>(whole.a.q) + k, p.b.q = static_cast<const uint8_t *>(whole.b.q) + k;
        p.a.s = whole.a.s + k / kFp8Block, p.b.s = whole.b.s + k / kFp8Block;
        if (k > 0) p.add = p.out, p.as = p.os;
        const cudaError_t e = launch_tile<E, BT>(args, sms, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Clusters of 4 and of 8 SMs of one part of the GPU that fit it: 36 and 15 of 152.
int64_t clusters_of_4(int sms) { return sms * 36 / 152; }
int64_t clusters_of_8(int sms) { return sms * 15 / 152; }

template <typename E, int BN, int SPLIT>
cudaError_t run_pair(MatmulArgs &args, int sms, cudaStream_t stream) {
    using S = PairShape<BN, SPLIT>;
    constexpr auto kernel = mm_pair_kernel<E, BN, SPLIT>;
    const cudaError_t e = allow_smem<kernel>(S::kSmem);
    if (e != cudaSuccess) return e;
    const MatmulParams &p = args.p;
    if (!encode_operand(args.a, p.a, p.K, kRows) || !encode_operand(args.b, p.b, p.K, BN / 2)) return cudaErrorInvalidValue;
    constexpr int V = 16 / sizeof(E);
    const auto aligned = [&](const void *t, int64_t stride, int n) { return reinterpret_cast<uintptr_t>(t) % (n * sizeof(E)) == 0 && stride % n == 0; };
    const int wide = !aligned(p.out, p.os, V) || (p.add && !aligned(p.add, p.as, V)) ? 0 : p.add && aligned(p.add, p.as, 2 * V) ? 2 : 1;
    if (SPLIT == 1 && wide && !encode_out(args.out, p)) return cudaErrorInvalidValue;
    constexpr int kCtas = 2 * SPLIT;
    const int64_t tiles = ceil_div(p.a.rows, 2 * kRows) * ceil_div(p.b.rows, BN), most = SPLIT > 1 ? tiles : sms / 2;
    return launch_early(kernel, kCtas * std::min(tiles, most), dim3(kPairThreads), S::kSmem, stream, kCtas, args, wide);
}

// How a product is computed: rows of a per tile (tile kernel), or rows of b and parts of K (pair
// kernel).
struct Choice {
    int bt, bn, split;
};

Choice choose(const MatmulParams &p, int sms) {
    if (p.a.rows <= 64) return {p.a.rows <= 16 ? 16 : p.a.rows <= 32 ? 32 : 64, 0, 0};
    const int64_t pairs = sms / 2, blocks = ceil_div(p.K, kFp8Block);
    Choice best = {};
    double least = 0;
    for (const Choice c : {Choice{0, 224, 1}, Choice{0, 192, 1}, Choice{0, 128, 1}, Choice{0, 256, 2}, Choice{0, 128, 2}, Choice{0, 128, 4}}) {
        if (p.dtype == kFP32 && c.bn == 224) continue;   // its sums do not fit the registers
        const int64_t tiles = ceil_div(p.a.rows, 2 * kRows) * ceil_div(p.b.rows, c.bn);
        if (c.split > 1 && (tiles > (c.split == 2 ? clusters_of_4(sms) : clusters_of_8(sms)) || blocks < 8 * c.split)) continue;
        // fp32 sums of a shared tile's part are not cut into segments
        if (c.split > 1 && p.dtype == kFP32 && blocks > c.split * kSegment) continue;
        // in cycles: an SM loads 64 bytes in one, (128 + bn / 2) * 128 for a block; the way into a
        // pipeline and out of it, and that of the parts through distributed shared memory
        const double cost = (256 + c.bn) * (c.split > 1 ? ceil_div(blocks, c.split) : ceil_div(tiles, pairs) * blocks) + (c.split > 1 ? 3500 : 0);
        if (best.bn && cost >= least) continue;
        least = cost;
        best = c;
    }
    return best;
}

// out = add, where K is 0.
template <typename E>
__global__ void __launch_bounds__(256) mm_add_kernel(MatmulParams p) {
    wait_for_prior_kernels();
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
            return launch_early(mm_add_kernel<E>, std::min(ceil_div(p.a.rows * p.b.rows, 256), (int64_t)sms * 8), dim3(256), 0, stream, 0, p);
        }
        const Choice c = choose(p, sms);
        MatmulArgs args;
        args.p = p;
        switch (c.bt) {
            case 16: return run_tile<E, 16>(args, sms, stream);
            case 32: return run_tile<E, 32>(args, sms, stream);
            case 64: return run_tile<E, 64>(args, sms, stream);
        }
        if (c.split == 4) return run_pair<E, 128, 4>(args, sms, stream);
        if (c.split == 2) return c.bn == 128 ? run_pair<E, 128, 2>(args, sms, stream) : run_pair<E, 256, 2>(args, sms, stream);
        if (c.bn == 128) return run_pair<E, 128, 1>(args, sms, stream);
        if (c.bn == 192) return run_pair<E, 192, 1>(args, sms, stream);
        if constexpr (sizeof(E) == 2) return run_pair<E, 224, 1>(args, sms, stream);
        return cudaErrorInvalidValue;
    });
}

}  // namespace kda
