// What the forward and the backward scan of the gated linear recurrence share: affine maps
// h -> A h + H and their products, the tiles, and the hand-over of a tile's map to the
// tiles after it.
//
// Both scans cut [rows, D] into tiles of 64 rows (a checkpoint's spacing) and one block of
// channels, and run as one cooperative launch of persistent CTAs: every CTA takes its tiles
// in ascending order, a tile waits only for tiles before it, and all CTAs are resident, so
// the first unfinished tile can always go on.  The tiles of a channel block form groups
// (scan_plan chooses their size).  A tile publishes its own map; it takes the state that enters it from the state
// after the previous group and the maps of its own group's earlier tiles, always the same
// ones in the same order, whatever has arrived first: the same bits every time.
// A published value is its own flag: the buffers are filled with ones (a NaN that is never
// published) before the launch.
#pragma once

#include <cooperative_groups.h>

#include "glr_gate.cuh"
#include "layer_copy.cuh"

namespace kda {
namespace layer {

constexpr uint32_t kEmpty = 0xffffffffu;

// An affine map.  A decay is never negative, so A's sign bit marks a map that does not
// depend on the state that enters it (a sequence begins inside): the state is left out,
// not multiplied by 0, and NaN and infinity stay within their sequence.
struct Affine { float A, H; };

__device__ __forceinline__ bool cuts(float A) { return __float_as_int(A) < 0; }
__device__ __forceinline__ float apply(Affine m, float h) { return cuts(m.A) ? m.H : fmaf(m.A, h, m.H); }
// First `a`, then `b`.  The product keeps the sign of a's A.
__device__ __forceinline__ Affine then(Affine a, Affine b) {
    return cuts(b.A) ? b : Affine{a.A * b.A, fmaf(b.A, a.H, b.H)};
}

// A NaN is published as the canonical one, so that no value looks empty.
__device__ __forceinline__ uint32_t bits_to_publish(float v) {
    return v == v ? __float_as_uint(v) : 0x7fffffffu;
}
__device__ __forceinline__ void publish(uint64_t *at, Affine m) {
    const uint64_t v = (uint64_t)bits_to_publish(m.H) << 32 | bits_to_publish(m.A);
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(at), "l"(v) : "memory");
}
__device__ __forceinline__ void publish(uint32_t *at, float h) {
    asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(at), "r"(bits_to_publish(h)) : "memory");
}
__device__ __forceinline__ uint64_t peek(const uint64_t *at) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t peek(const uint32_t *at) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
    return v;
}
__device__ __forceinline__ bool empty(uint64_t v) { return (uint32_t)v == kEmpty; }
__device__ __forceinline__ bool empty(uint32_t v) { return v == kEmpty; }

// What the waits of a CTA report to: the device error word, and a flag in the CTA's shared
// memory (0 at first) that its first expired wait sets.  After that its waits are short, so
// that the kernel ends soon however much is missing.  On expiry a wait goes on with what is
// there.
struct Waits { int *err; volatile int *late; };
__device__ __forceinline__ void expire(const Waits &w) {
    atomicExch(w.err, kErrTimeout);
    *w.late = 1;
}

// Waits until `all_there`, which looks again at what is missing, says so; at most kWaitPolls
// looks (about a second).  One loop for all the values of a batch: one for each of them took
// 237 us in the backward pass of 8192 x 8192 bf16, so 230.
constexpr int kWaitPolls = 1 << 22, kLatePolls = 1 << 10;
template <typename F>
__device__ __forceinline__ void await(const Waits &w, F &&all_there) {
    for (int polls = 0; !all_there(); ++polls) {
        if (polls < kWaitPolls && !(polls > kLatePolls && *w.late)) continue;
        expire(w);
        break;
    }
}
// One published value, of which v is the first look.
template <typename U>
__device__ __forceinline__ U await(const Waits &w, const U *at, U v) {
    if (empty(v)) await(w, [&] { return !empty(v = peek(at)); });
    return v;
}

// Waits for a tile's copies.
constexpr uint64_t kCopyWaitNs = 2000000000ull, kLateCopyNs = 1000000ull;
__device__ __forceinline__ void wait_copies(uint64_t *arrived, uint32_t parity, const Waits &w) {
    if (sm103::mbar_try_wait(arrived, parity)) return;
    const uint64_t end = sm103::globaltimer_ns() + (*w.late ? kLateCopyNs : kCopyWaitNs);
    while (!sm103::mbar_try_wait(arrived, parity)) {
        if (sm103::globaltimer_ns() < end) continue;
        expire(w);
        break;
    }
}

// How a CTA covers a tile: THREADS threads as CL channel lanes of V channels each by RG row
// groups of L rows each.
template <int ROWS_, int THREADS_, int CL_, int V_>
struct TileShape {
    static constexpr int ROWS = ROWS_, THREADS = THREADS_, CL = CL_, V = V_;
    static constexpr int CB = CL * V, RG = THREADS / CL, L = ROWS / RG;
    static_assert(RG * L == ROWS && THREADS >= 2 * CB && CB % 32 == 0, "tile shape");
};

// One input of a tile in shared memory.  From aligned rows (TMA) a box of a tensor map.
// Other rows come as whole 16-byte granules, so that a row begins at its first element's
// place in a granule (RowStart) and takes up to one granule more.  PHASES rows apart that
// place is the same: these rows lie together, and a tensor map of theirs has a legal pitch.
// (A bulk copy per row instead was as fast in the 16-bit backward pass, but 115 us against
// 99 in the forward one, 8192 x 3937 bf16, and 238 against then 201 on 20011 x 847 fp32
// backward.)
template <typename E, typename S, bool TMA>
struct RawTile {
    static constexpr int PHASES = TMA ? 1 : 16 / (int)sizeof(E), PITCH = S::CB + (TMA ? 0 : PHASES), EACH = S::ROWS / PHASES;
    E e[PHASES][EACH][PITCH];
    static_assert(S::L % PHASES == 0 || PHASES % S::L == 0, "a row group's phases follow each other");
    // row r of a row group
    __device__ __forceinline__ E *row(int rg, int r) {
        return &e[rg * S::L % PHASES][rg * S::L / PHASES][0] + (r % PHASES * EACH + r / PHASES) * PITCH;
    }
    __device__ __forceinline__ Pack<E, S::V> &at(int rg, int r, int lane) { return *reinterpret_cast<Pack<E, S::V> *>(row(rg, r) + lane * S::V); }
};
template <typename E>
struct RowStart {
    uint32_t first, step;
    __device__ __forceinline__ RowStart(const void *p, int64_t stride)
        : first((uint32_t)(reinterpret_cast<uintptr_t>(p) / sizeof(E))), step((uint32_t)stride) {}
    // of a row of a tile (tiles begin at multiples of 64 rows)
    __device__ __forceinline__ int operator[](int row) const { return (first + (uint32_t)row * step) & (16 / sizeof(E) - 1); }
};
// Tensor maps of a tile's N inputs.  Not `boxed`: without them (rows that overlap, as of a
// broadcast tensor, and too few rows for the phases).
template <int N>
struct ScanMaps {
    CUtensorMap m[N];
    int boxed;
};
// The maps begin at a whole granule, which is inside the allocation, and end with the rows'
// last element: nothing else is read.
template <typename Raw, int N>
bool encode_maps(ScanMaps<N> &maps, int k, const void *ptr, int64_t stride, int64_t rows, int64_t D, int dtype) {
    const int64_t e = (int64_t)dtype_bytes(dtype);
    for (int ph = 0; ph < Raw::PHASES; ++ph) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(ptr) + ph * stride * e, floor = at / 16 * 16;
        if (!encode_tile_map(maps.m[k * Raw::PHASES + ph], reinterpret_cast<const void *>(floor), Raw::PHASES * stride,
                             (rows - ph + Raw::PHASES - 1) / Raw::PHASES, (int64_t)(at - floor) / e + D, dtype, Raw::PITCH, Raw::EACH))
            return false;
    }
    return true;
}
// Starts the boxes of a tile, by one thread or, of several phases, one to a lane of the CTA's
// first warp; `bytes` more are to arrive with them.  (Copies of 8 bytes per thread and row
// took a fifth of a tile's time to issue: 119 us forward and 289 us backward on 8192 x 8192
// bf16.)
template <typename Raw, int N, int M>
__device__ __forceinline__ void fetch_boxes(Raw (&raw)[N], const ScanMaps<M> &maps, int64_t r0, int c, uint32_t bytes, uint64_t *arrived) {
    static_assert(M == N * Raw::PHASES && M <= 32, "a box per lane");
    if constexpr (Raw::PHASES == 1) {
        if (threadIdx.x != 0) return;
        sm103::mbar_arrive_expect_tx(arrived, bytes + sizeof(raw));
#pragma unroll
        for (int k = 0; k < N; ++k) tma_box(raw[k].e, maps.m[k], arrived, c, (int)r0);
        return;
    }
    if (threadIdx.x >= 32) return;
    if (threadIdx.x == 0) sm103::mbar_arrive_expect_tx(arrived, bytes + sizeof(raw));
    __syncwarp();
    if (threadIdx.x < M)
        tma_box(raw[threadIdx.x / Raw::PHASES].e[threadIdx.x % Raw::PHASES], maps.m[threadIdx.x], arrived, c, (int)(r0 / Raw::PHASES));
}
// V elements from any place of a row in shared memory.
template <typename E, int V>
__device__ __forceinline__ Pack<E, V> pick(const E *row, int at) {
    Pack<E, V> t;
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int v = 0; v < V; ++v) t.e[v] = row[at + v];
    } else {
        static_assert(V == 4, "two words");
        const uint32_t *w = reinterpret_cast<const uint32_t *>(row) + (at >> 1);
        const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], by = (at & 1) * 16;
        uint32_t *to = reinterpret_cast<uint32_t *>(t.e);
        to[0] = __funnelshift_r(w0, w1, by);
        to[1] = __funnelshift_r(w1, w2, by);
    }
    return t;
}
// Without maps: the elements one by one.  Every thread arrives, with `bytes` more to come.
template <typename E, typename S, int N>
__device__ __forceinline__ void fetch_elements(RawTile<E, S, false> (&raw)[N], const void *const (&src)[N], const int64_t (&stride)[N],
                                               int64_t rows, int64_t D, int64_t r0, int c, uint32_t bytes, uint64_t *arrived) {
    using Raw = RawTile<E, S, false>;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const RowStart<E> start(src[k], stride[k]);
#pragma unroll 4
        for (int j = threadIdx.x; j < S::ROWS * S::CB; j += S::THREADS) {
            const int row = j / S::CB, m = j % S::CB;
            if (r0 + row < rows && c + m < D)
                raw[k].e[row % Raw::PHASES][row / Raw::PHASES][start[row] + m] = static_cast<const E *>(src[k])[(r0 + row) * stride[k] + c + m];
        }
    }
    sm103::fence_proxy_async_smem();
    sm103::mbar_arrive_expect_tx(arrived, bytes);
}

// Workspace of a scan and its tiles.  Maps [row tile][padded channel], states after a
// group [group][padded channel], then the first sequence of every row tile.
struct ScanPlan {
    int64_t row_tiles, groups, blocks, width;   // width = blocks * channels per block
    int tile_rows, group_log2;                  // rows per tile, log2 of row tiles per group
    uint64_t *maps;
    uint32_t *states;
    int *first_seq;                             // kInside set: the tile lies inside that sequence
    GateConst *gates;                           // [width]
};
constexpr int kInside = INT32_MIN;
template <typename S>
ScanPlan scan_plan(int64_t rows, int64_t D, unsigned char *ws, size_t *bytes) {
    ScanPlan s;
    s.tile_rows = S::ROWS;
    s.row_tiles = ceil_div(rows, S::ROWS);
    s.blocks = ceil_div(D, S::CB);
    // The state passes from group to group one at a time, each step about one tile's time
    // on one SM, while the rest of the GPU works off `group` row tiles of `blocks` tiles; a
    // tile joins the maps of half a group on average.
    for (s.group_log2 = 2; s.group_log2 < 5 && s.blocks << s.group_log2 < 256; ++s.group_log2) {}
    s.groups = ceil_div(s.row_tiles, int64_t(1) << s.group_log2);
    s.width = s.blocks * S::CB;
    s.maps = reinterpret_cast<uint64_t *>(ws);
    s.states = reinterpret_cast<uint32_t *>(s.maps + s.row_tiles * s.width);
    s.gates = reinterpret_cast<GateConst *>(s.states + ceil_div(s.groups * s.width, 4) * 4);
    s.first_seq = reinterpret_cast<int *>(s.gates + s.width);
    if (bytes) *bytes = (size_t)(reinterpret_cast<unsigned char *>(s.first_seq + s.row_tiles) - ws + 15) / 16 * 16;
    return s;
}

// The first part of a scan kernel, before its grid-wide barrier: empties the hand-over
// buffers, folds the gates' constants, finds the first sequence of every row tile.  REVERSE
// false: final states of sequences without tokens; true: their gradients of the initial
// state.  (As a kernel of its own it cost 4 us and a launch.)
template <bool UB, bool REVERSE>
__device__ __forceinline__ void prepare_scan(const GlrParams &p, const ScanPlan &s) {
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    const int64_t words = (s.row_tiles * s.width * 2 + ceil_div(s.groups * s.width, 4) * 4) / 4;
    uint4 *fill = reinterpret_cast<uint4 *>(s.maps);
    for (int64_t j = at; j < words; j += step) fill[j] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    for (int64_t c = at; c < s.width; c += step)
        s.gates[c] = c < p.D ? gate_const<UB>(p.A_log[(unsigned)c / (unsigned)p.K], p.dt_bias[c]) : GateConst{0.f, 0.f};
    for (int64_t t = at; t < s.row_tiles; t += step) {
        const int64_t r0 = t * s.tile_rows, n = p.cu_seqlens ? seq_of_row(p.cu_seqlens, p.N, r0) : (unsigned)r0 / (unsigned)p.T;
        int64_t lo, hi;
        seq_rows(p, n, lo, hi);
        s.first_seq[t] = (int)n | (lo < r0 && hi > r0 + s.tile_rows ? kInside : 0);
    }
    if (!p.cu_seqlens && p.T > 0) return;
    if (REVERSE ? !p.dinit : !p.fin) return;
    // a warp per sequence: one without tokens passes its state through
    for (int64_t n = at >> 5; n < p.N; n += step >> 5) {
        int64_t lo, hi;
        seq_rows(p, n, lo, hi);
        if (lo < hi) continue;
        for (int64_t c = n * p.D + (threadIdx.x & 31); c < (n + 1) * p.D; c += 32) {
            if (REVERSE) p.dinit[c] = p.dfinal ? p.dfinal[c] : 0.f;
            else st_state(p.fin, p.state_type, c, p.init ? ld_state(p.init, p.state_type, c) : 0.f);
        }
    }
}

// A thread's gate constants, one array each.
template <int V>
struct ChannelGates {
    float k0[V], k1[V];
    __device__ __forceinline__ ChannelGates(const Pack<GateConst, V> &g) {
#pragma unroll
        for (int v = 0; v < V; ++v) k0[v] = g.e[v].k0, k1[v] = g.e[v].k1;
    }
};

// One map after the other where neither cuts.
template <bool CUTS>
__device__ __forceinline__ Affine joined(Affine a, Affine b) {
    return CUTS ? then(a, b) : Affine{a.A * b.A, fmaf(b.A, a.H, b.H)};
}
template <bool CUTS>
__device__ __forceinline__ float applied(Affine m, float h) { return CUTS ? apply(m, h) : fmaf(m.A, h, m.H); }

// One channel's maps of a tile's row groups, loaded together: the joins that follow are a
// chain, and a shared-memory load in each of its links made it five times as long.
template <int RG, int CL, int V>
struct GroupMaps {
    Affine m[RG];
    __device__ __forceinline__ GroupMaps(const Pack<float, V> (&A)[RG][CL], const Pack<float, V> (&H)[RG][CL], int ch) {
#pragma unroll
        for (int q = 0; q < RG; ++q) m[q] = Affine{A[q][ch / V].e[ch % V], H[q][ch / V].e[ch % V]};
    }
};

// Where sequences begin and end within a tile of rows [r0, r0 + ROWS): for each row
// the sequence that it begins (ends), or -1.  Returns false, and writes nothing, where the
// tile lies inside one sequence.  Called by all threads, whose shared memory it is.
template <int ROWS> struct TileMarks { int begins[ROWS], ends[ROWS]; };

// n: first_seq of the tile.
template <typename P, int ROWS>
__device__ __forceinline__ bool mark_tile(const P &p, int64_t row_tile, int n, TileMarks<ROWS> &m) {
    if (n & kInside) return false;
    const int64_t r0 = row_tile * ROWS, r1 = r0 + ROWS;
    __syncthreads();   // the marks of the tile before are read no more
    if (threadIdx.x < ROWS) m.begins[threadIdx.x] = m.ends[threadIdx.x] = -1;
    __syncthreads();
    for (int64_t k = n + threadIdx.x; k < p.N; k += blockDim.x) {
        int64_t lo, hi;
        seq_rows(p, k, lo, hi);
        if (lo >= r1) break;
        if (lo >= hi) continue;
        if (lo >= r0) m.begins[lo - r0] = (int)k;
        if (hi > r0 && hi <= r1) m.ends[hi - 1 - r0] = (int)k;
    }
    __syncthreads();
    return true;
}

// The maps of `count` row tiles of a channel, one after the other, as one map.  `at` is the
// first one's, the next `stride` further on; kBatch are in flight together.  Forward 4: 8
// spill there (8192 x 8192 bf16 101.5 and 103.6 us, without a lower bound 111.8 and 114.7),
// though they help where channels are few (65536 x 256: 48.5 and 45.3 us).  Backward 8: 230
// and 243 us, 65536 x 1024 270 and 293.
template <int kBatch = 8>
__device__ __forceinline__ Affine join_maps(const uint64_t *at, int64_t stride, int count, const Waits &waits) {
    Affine t{1.f, 0.f};
    for (int j0 = 0; j0 < count; j0 += kBatch, at += kBatch * stride) {
        uint64_t w[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) w[j] = j0 + j < count ? peek(at + j * stride) : 0x3f800000ull;   // (1, 0)
        bool there = true;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) there &= !empty(w[j]);
        if (!there) {
            await(waits, [&] {
                bool all = true;
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (empty(w[j])) w[j] = peek(at + j * stride);
                    all &= !empty(w[j]);
                }
                return all;
            });
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            t = then(t, Affine{__uint_as_float((uint32_t)w[j]), __uint_as_float((uint32_t)(w[j] >> 32))});
        }
    }
    return t;
}

// Tiles of a persistent CTA: row tile and channel block, stepped by the grid's size.
struct TileWalk {
    int64_t rt;
    int cb, blocks, step_rt, step_cb;
    __device__ __forceinline__ TileWalk(const ScanPlan &s) {
        blocks = (int)s.blocks;
        rt = blockIdx.x / (unsigned)blocks;
        cb = (int)(blockIdx.x % (unsigned)blocks);
        step_rt = (int)(gridDim.x / (unsigned)blocks);
        step_cb = (int)(gridDim.x % (unsigned)blocks);
    }
    __device__ __forceinline__ void next() {
        rt += step_rt;
        cb += step_cb;
        if (cb >= blocks) cb -= blocks, ++rt;
    }
};

// CTAs of a kernel that an SM holds, its dynamic shared memory allowed first; looked up once
// per device.
template <auto Kernel>
cudaError_t resident_ctas(int threads, int smem, int &ctas) {
    static std::atomic<bool> done[kMaxDevices];
    static int per_sm[kMaxDevices];
    int dev = 0;
    ctas = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once_per_device(done, [&](int d) {
        cudaError_t r = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r == cudaSuccess) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, Kernel, threads, smem);
        if (r == cudaSuccess && ctas < 1) r = cudaErrorInvalidConfiguration;
        if (d < kMaxDevices) per_sm[d] = ctas;
        return r;
    });
    if (dev < kMaxDevices) ctas = per_sm[dev];
    return e;
}

}  // namespace layer
}  // namespace kda
