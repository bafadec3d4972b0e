// Gated linear recurrence, backward.  With e_t the gradient of h_t and f_t = a_t e_t what
// passes on to h_{t-1},
//   e_t = dout_t + f_{t+1}   (of a sequence's last token also + dfinal)
//   f_t = a_t f_{t+1} + a_t dout_t
//   dx = e s, di = e x s (1 - s), s = sigma(i);   dl = f_t h_{t-1}, the gradient of gk_t;
//   dg = dl d gk/dg, ddt_bias = sum dg, dA_log = sum dl d gk/dA_log, dinit = f_first.
//
// One pass over tiles of 64 rows from the last to the first (glr_scan.cuh).  h_{t-1} is
// recomputed in fp32: a tile's rows are those of one checkpoint, so the forward states need
// no other tile.  A thread forms the decays of its elements and folds them forward (from
// the checkpoint) and backward (into the map that the tile hands on); with the states that
// enter its rows from both sides it then forms the gradients, the inputs still in shared
// memory and three values per element in registers.  The slopes of saturated gates are exact
// relative to themselves: no 1 - sigma is taken of a sigma near 1.  Inputs are read and
// gradients written once.  Parameter gradients leave a tile as one partial sum per channel.
#include <algorithm>

#include "glr_scan.cuh"

namespace kda {
namespace {

using namespace layer;

// 16 bits: 4 rows by 4 channels per thread, 2 CTAs per SM (the raw inputs of two tiles each
// in shared memory).  32 bits: 8 rows by 2 channels and 3 CTAs of 128 threads (65536 x 1024:
// 326 us, 2 CTAs of 256 363; 8192 x 8192: 315 and 309, without a lower bound 318 and 340).
// There the granules of unaligned rows leave room for 2 CTAs only, so they have 256 threads of
// 4 rows: 20011 x 847 171 us, with 128 threads 190.
// 8192 x 8192 bf16: 228 us, 4.1 TB/s; what bounds it is issue, 75 instructions per element
// between barriers, at 59% of the slots.  Unaligned: 8192 x 3937 bf16 250 us (aligned 3968:
// 125 us); element-wise copies took 475 us, and 214 us on 20011 x 847 fp32.
template <typename E, bool TMA>
using BwdShape = TileShape<kGlrCheckpointRows, sizeof(E) == 2 || !TMA ? 256 : 128, 16, sizeof(E) == 2 ? 4 : 2>;

template <typename E, bool TMA>
struct BwdShared {
    using S = BwdShape<E, TMA>;
    RawTile<E, S, TMA> raw[2][4];                                  // x, i, g, dout
    Pack<GateConst, S::V> gates[2][S::CL];
    Pack<float, S::V> A[S::RG][S::CL], H[S::RG][S::CL];            // forward maps of the row groups
    Pack<float, S::V> B[S::RG][S::CL], F[S::RG][S::CL];            // backward maps
    // states that enter them, and over each thread's own two its sums of parameter gradients
    Pack<float, S::V> h[S::RG][S::CL], f[S::RG][S::CL];
    TileMarks<S::ROWS> marks;
    uint64_t arrived[2];                                           // of a tile's copies
    int late;
};

template <typename E, bool TMA, bool UB>
__global__ void __launch_bounds__(BwdShape<E, TMA>::THREADS, sizeof(E) == 2 || !TMA ? 2 : 3)
    glr_bwd_scan_kernel(GlrParams p, ScanPlan s, const __grid_constant__ ScanMaps<4 * RawTile<E, BwdShape<E, TMA>, TMA>::PHASES> maps,
                        float *part_ddt, float *part_dA) {
    using namespace sm103;
    using S = BwdShape<E, TMA>;
    constexpr int CL = S::CL, V = S::V, L = S::L, CB = S::CB, RG = S::RG;
    static_assert(S::THREADS >= 3 * CB, "roles");
    extern __shared__ __align__(128) unsigned char smem[];
    BwdShared<E, TMA> &sh = *reinterpret_cast<BwdShared<E, TMA> *>(smem);
    const int tid = threadIdx.x, lane = tid % CL, rg = tid / CL;
    const int role = tid / CB, ch = tid % CB, D = (int)p.D;
    const float lb2 = p.lower_bound * kLog2e;
    float checkpoint = 0.f;   // of role 2's channel, fetched with the tile

    // starts the copies of a tile's inputs; tile number w.rt counts from the last row tile
    const auto fetch = [&](const TileWalk &w, int stage) {
        if (w.rt >= s.row_tiles) return;
        const int64_t rt = s.row_tiles - 1 - w.rt;
        if (role == 2 && w.cb * CB + ch < D) checkpoint = p.checkpoints[rt * p.D + w.cb * CB + ch];
        if (TMA || maps.boxed) {
            fetch_boxes(sh.raw[stage], maps, rt * S::ROWS, w.cb * CB, sizeof(sh.gates[0]), &sh.arrived[stage]);
        } else if constexpr (!TMA) {
            fetch_elements<E, S, 4>(sh.raw[stage], {p.x, p.i, p.g, p.dout}, {p.xs, p.is, p.gs, p.ds}, p.rows, p.D, rt * S::ROWS,
                                    w.cb * CB, tid == 0 ? sizeof(sh.gates[0]) : 0, &sh.arrived[stage]);
        }
    };
    // and of what the scan's first part has left for the tile; returns its first sequence
    const auto fetch_plan = [&](const TileWalk &w, int stage) {
        int first = 0;
        if (w.rt < s.row_tiles) {
            first = s.first_seq[s.row_tiles - 1 - w.rt];
            const GateConst *gates = s.gates + w.cb * CB;
            if (tid == 0) bulk_load(smem_u32(sh.gates[stage]), gates, sizeof(sh.gates[0]), smem_u32(&sh.arrived[stage]));
        }
        return first;
    };
    const Waits waits{p.err, &sh.late};
    const RowStart<E> starts[4] = {{p.x, p.xs}, {p.i, p.is}, {p.g, p.gs}, {p.dout, p.ds}};

    if (tid == 0) {
        mbar_init(&sh.arrived[0], TMA || maps.boxed ? 1 : S::THREADS);
        mbar_init(&sh.arrived[1], TMA || maps.boxed ? 1 : S::THREADS);
        sh.late = 0;
        fence_mbar_init();
    }
    __syncthreads();
    TileWalk w(s);
    fetch(w, 0);
    prepare_scan<UB, true>(p, s);
    fence_proxy_async_global();   // the gates are read by bulk copies
    cooperative_groups::this_grid().sync();
    fence_proxy_async_global();
    int next_first = fetch_plan(w, 0);
    uint32_t parity = 0;   // of stage 0's copies; stage 1's turn comes in between
    for (int stage = 0; w.rt < s.row_tiles; stage ^= 1) {
        const int64_t walk = w.rt, rt = s.row_tiles - 1 - walk, r0 = rt * S::ROWS + rg * L;
        const int c = w.cb * CB + lane * V, block = w.cb * CB, cols = D - c, first = next_first;
        const float h_tile = checkpoint;
        w.next();
        fetch(w, stage ^ 1);
        next_first = fetch_plan(w, stage ^ 1);
        const bool marked = mark_tile(p, rt, first, sh.marks);
        const bool plain = !marked && (rt + 1) * S::ROWS <= p.rows;        // every row inside one sequence
        const int left = cols > 0 ? (int)min(p.rows - r0, (int64_t)L) : 0;   // rows of this thread that exist
        wait_copies(&sh.arrived[stage], parity, waits);
        parity ^= stage;
        if constexpr (!TMA) {
            // each row to its aligned place, as it is read several times (15 us of 185 on
            // 8192 x 3968 bf16); the lanes of a row are in one warp
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                Pack<E, V> t[L];
#pragma unroll
                for (int r = 0; r < L; ++r) t[r] = pick<E, V>(sh.raw[stage][k].row(rg, r), starts[k][rg * L + r] + lane * V);
                __syncwarp();
#pragma unroll
                for (int r = 0; r < L; ++r) sh.raw[stage][k].at(rg, r, lane) = t[r];
            }
            fence_proxy_async_smem();   // before the copies that follow this tile
        }

        const ChannelGates<V> gc(sh.gates[stage][lane]);
        const auto raw = [&](int k, int r, float (&f)[V]) { unpack<E, V>(sh.raw[stage][k].at(rg, r, lane), f); };
        float a[L][V], si[L][V], kept[L][V];   // for the second half: decays, sigma(i), the gates' slopes
        Pack<float, V> mA, mH, mB, mF;
#pragma unroll
        for (int v = 0; v < V; ++v) mA.e[v] = mB.e[v] = 1.f, mH.e[v] = mF.e[v] = 0.f;
        if (plain) {
#pragma unroll
            for (int r = 0; r < L; ++r) {
                float x[V], i[V], g[V], d[V], sx[V];
                raw(0, r, x), raw(1, r, i), raw(2, r, g), raw(3, r, d);
                sigmoid_n<V>(si[r], i);
                decay_and_kept_n<UB, V>(a[r], kept[r], g, gc.k0, gc.k1, lb2);
                mul_n<V>(sx, si[r], x);
                // forward: after the rows before; backward: f = a_0 (dout_0 + a_1 (dout_1 + ...))
                fma_n<V>(mH.e, a[r], mH.e, sx);
                mul_n<V>(mA.e, a[r], mA.e);
                fma_n<V>(mF.e, mA.e, d, mF.e);
            }
            mB = mA;
        } else {
#pragma unroll 1
            for (int r = 0; r < left; ++r) {
                float x[V], i[V], g[V], d[V], sx[V], ar[V], sr[V], kr[V];
                raw(0, r, x), raw(1, r, i), raw(2, r, g), raw(3, r, d);
                sigmoid_n<V>(sr, i);
                decay_and_kept_n<UB, V>(ar, kr, g, gc.k0, gc.k1, lb2);
                mul_n<V>(sx, sr, x);
                const int begins = marked ? sh.marks.begins[rg * L + r] : -1, ends = marked ? sh.marks.ends[rg * L + r] : -1;
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int k = 0; k < L; ++k)
                        if (k == r) a[k][v] = ar[v], si[k][v] = sr[v], kept[k][v] = kr[v];
                    if (begins >= 0) {
                        const float h0 = p.init && v < cols ? ld_state(p.init, p.state_type, begins * p.D + c + v) : 0.f;
                        mA.e[v] = -0.f, mH.e[v] = fmaf(ar[v], h0, sx[v]);
                    } else {
                        mH.e[v] = fmaf(ar[v], mH.e[v], sx[v]);
                        mA.e[v] *= ar[v];
                    }
                    // backward map of rows 0 .. r: the earlier rows' map after this row's
                    const float dt = ends >= 0 && p.dfinal && v < cols ? d[v] + p.dfinal[ends * p.D + c + v] : d[v];
                    const Affine m = then(Affine{ends >= 0 ? -0.f : ar[v], ar[v] * dt}, Affine{mB.e[v], mF.e[v]});
                    mB.e[v] = m.A, mF.e[v] = m.H;
                }
            }
        }
        sh.A[rg][lane] = mA;
        sh.H[rg][lane] = mH;
        sh.B[rg][lane] = mB;
        sh.F[rg][lane] = mF;
        __syncthreads();

        const int64_t group = walk >> s.group_log2;
        const int pos = (int)(walk - (group << s.group_log2)), last = (1 << s.group_log2) - 1;
        if (role == 0) {
            // the tile's backward map, handed on
            if (pos != last) {
                const GroupMaps<RG, CL, V> back(sh.B, sh.F, ch);
                Affine t = back.m[RG - 1];
                if (plain) {
#pragma unroll
                    for (int q = RG - 2; q >= 0; --q) t = joined<false>(t, back.m[q]);
                } else {
#pragma unroll
                    for (int q = RG - 2; q >= 0; --q) t = joined<true>(t, back.m[q]);
                }
                publish(s.maps + walk * s.width + block + ch, t);
            }
        } else if (role == 1) {
            // what enters the tile and its row groups from behind
            const uint32_t *before = s.states + (group - 1) * s.width + block + ch;
            const uint32_t f_bits = group > 0 ? peek(before) : 0;
            const Affine t = join_maps(s.maps + (walk - pos) * s.width + block + ch, s.width, pos, waits);
            float f = apply(t, group > 0 ? __uint_as_float(await(waits, before, f_bits)) : 0.f);
            const GroupMaps<RG, CL, V> back(sh.B, sh.F, ch);
#pragma unroll
            for (int q = RG - 1; q >= 0; --q) {
                sh.f[q][ch / V].e[ch % V] = f;
                f = plain ? applied<false>(back.m[q], f) : applied<true>(back.m[q], f);
            }
            if (pos == last) publish(s.states + group * s.width + block + ch, f);
        } else if (role == 2) {
            // the forward states that enter the row groups
            const GroupMaps<RG, CL, V> fore(sh.A, sh.H, ch);
            float h = h_tile;
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                sh.h[q][ch / V].e[ch % V] = h;
                h = plain ? applied<false>(fore.m[q], h) : applied<true>(fore.m[q], h);
            }
        }
        __syncthreads();

        Pack<float, V> ddt, dA;
#pragma unroll
        for (int v = 0; v < V; ++v) ddt.e[v] = dA.e[v] = 0.f;
        float h[V], f[V];
        const Pack<float, V> h_in = sh.h[rg][lane], f_in = sh.f[rg][lane];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = h_in.e[v], f[v] = f_in.e[v];
        const int64_t row_at = r0 * p.D + c;
        // the state after a row from the one before it
        const auto advance = [&](int r) {
            float x[V];
            raw(0, r, x);
            mul_n<V>(x, si[r], x);
            fma_n<V>(h, a[r], h, x);
        };
        // the gradients of a row from its state `start` and what comes from behind
        const auto row = [&](int r, const float (&start)[V]) {
            float x[V], i[V], g[V], grad[V], o[V], out[V], slope[V], rate[V];
            raw(0, r, x), raw(2, r, g), raw(3, r, grad);
            add_n<V>(grad, grad, f);
            mul_n<V>(f, a[r], grad);
            mul_n<V>(out, grad, si[r]);
            st_cols<E, V, TMA>(static_cast<E *>(p.dx) + row_at + r * p.D, out, cols);
            raw(1, r, i);
            sigmoid_n<V>(o, i, kLog2e);   // sigma(-i) anew, exact relative to itself as 1 - sigma(i) is not
            mul_n<V>(out, out, o);
            mul_n<V>(out, out, x);
            st_cols<E, V, TMA>(static_cast<E *>(p.di) + row_at + r * p.D, out, cols);
            gate_slopes_n<UB, V>(slope, rate, g, kept[r], gc.k0, gc.k1, p.lower_bound);
            mul_n<V>(o, f, start);        // the gradient of gk
            mul_n<V>(out, o, slope);
            st_cols<E, V, TMA>(static_cast<E *>(p.dg) + row_at + r * p.D, out, cols);
            add_n<V>(ddt.e, ddt.e, out);
            fma_n<V>(dA.e, o, rate, dA.e);
        };
        if (plain) {
            if (cols > 0) {
                // The states that the rows start from; of 4 rows over the thread's own maps, which
                // nobody reads any more, as registers are short.
                Pack<float, V> *const slots[4] = {&sh.A[rg][lane], &sh.H[rg][lane], &sh.B[rg][lane], &sh.F[rg][lane]};
                float start[L][V];
#pragma unroll
                for (int r = 0; r < L; ++r) {
#pragma unroll
                    for (int v = 0; v < V; ++v) start[r][v] = h[v];
                    if constexpr (L == 4) st_f<float, V>(slots[r]->e, h);
                    if (r < L - 1) advance(r);
                }
#pragma unroll
                for (int r = L - 1; r >= 0; --r) {
                    if constexpr (L == 4) ld_f<float, V>(slots[r]->e, start[r]);
                    row(r, start[r]);
                }
            }
        } else {
            float start[L][V];
#pragma unroll
            for (int r = 0; r < L; ++r) {
                if (r >= left) break;
                const int begins = marked ? sh.marks.begins[rg * L + r] : -1;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (begins >= 0) h[v] = p.init && v < cols ? ld_state(p.init, p.state_type, begins * p.D + c + v) : 0.f;
                    start[r][v] = h[v];
                }
                advance(r);
            }
#pragma unroll
            for (int r = L - 1; r >= 0; --r) {
                if (r >= left) continue;
                const int ends = marked ? sh.marks.ends[rg * L + r] : -1, begins = marked ? sh.marks.begins[rg * L + r] : -1;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (ends >= 0) f[v] = p.dfinal && v < cols ? p.dfinal[ends * p.D + c + v] : 0.f;
                row(r, start[r]);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (begins >= 0 && p.dinit && v < cols) p.dinit[begins * p.D + c + v] = f[v];
            }
        }
        sh.h[rg][lane] = ddt;
        sh.f[rg][lane] = dA;
        __syncthreads();
        if (role < 2) {
            const auto &sum = role == 0 ? sh.h : sh.f;
            float t = 0.f;
#pragma unroll
            for (int q = 0; q < RG; ++q) t += sum[q][ch / V].e[ch % V];
            (role == 0 ? part_ddt : part_dA)[rt * s.width + block + ch] = role == 0 ? t : t * rate_unit<UB>(p.lower_bound);
        }
    }
}

// Sums the tiles' partial parameter gradients [parts, width] over the tiles: a CTA per head
// of at most 512 channels, ddt_bias per channel and dA_log; 1024 threads, as many slices of
// the parts as they allow.
constexpr int64_t kMaxHead = 512;
__global__ void __launch_bounds__(1024) glr_head_grads_kernel(GlrParams p, int64_t parts, int64_t width, const float *part_ddt,
                                                              const float *part_dA) {
    __shared__ float sums[2][1024];
    const int K = (int)p.K, lanes = (K + 31) / 32 * 32, slices = lanes > 0 ? 1024 / lanes : 0;
    const int k = lanes > 0 ? threadIdx.x % lanes : 0, slice = lanes > 0 ? threadIdx.x / lanes : 0;
    const int64_t c = blockIdx.x * p.K + k;
    float ddt = 0.f, dA = 0.f;
    if (k < K && slice < slices) {
#pragma unroll 8
        for (int64_t j = slice; j < parts; j += slices) {
            ddt += part_ddt[j * width + c];
            dA += part_dA[j * width + c];
        }
    }
    sums[0][threadIdx.x] = ddt;
    sums[1][threadIdx.x] = dA;
    __syncthreads();
    ddt = dA = 0.f;
    if (threadIdx.x < K) {
        for (int j = 0; j < slices; ++j) ddt += sums[0][j * lanes + k], dA += sums[1][j * lanes + k];
        p.ddt_bias[c] = ddt;
    }
    __syncthreads();
    for (int o = 16; o; o >>= 1) dA += __shfl_xor_sync(0xffffffffu, dA, o);
    if ((threadIdx.x & 31) == 0) sums[0][threadIdx.x >> 5] = dA;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int j = 1; j < 32; ++j) dA += sums[0][j];
        p.dA_log[blockIdx.x] = dA;
    }
}
// Wider heads: the sums per channel first, 32 channels per CTA, those of dA_log left in
// part_dA's first row; then a CTA per head.
__global__ void __launch_bounds__(kSumThreads) glr_param_sum_kernel(GlrParams p, int64_t parts, int64_t width, const float *part_ddt,
                                                                    float *part_dA) {
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const float ddt = column_sum(part_ddt, parts, width, c, c < p.D);
    __syncthreads();
    const float dA = column_sum(part_dA, parts, width, c, c < p.D);
    if (threadIdx.x < 32 && c < p.D) {
        p.ddt_bias[c] = ddt;
        if (parts > 0) part_dA[c] = dA;   // no other CTA reads this column
    }
}
__global__ void __launch_bounds__(128) glr_head_sum_kernel(GlrParams p, bool any, const float *dA) {
    __shared__ float sums[4];
    float t = 0.f;
    if (any)
        for (int64_t k = threadIdx.x; k < p.K; k += 128) t += dA[blockIdx.x * p.K + k];
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) p.dA_log[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// The forward run that writes checkpoints only.
GlrParams states_only(const GlrParams &p) {
    GlrParams f = p;
    f.out = f.fin = nullptr;
    return f;
}

// Rows that tensor maps take, and gradients that allow stores of a thread's groups.
bool aligned_rows(const GlrParams &p) {
    const size_t e = dtype_bytes(p.dtype);
    return tma_rows(p.x, p.xs, p.D, e) && tma_rows(p.i, p.is, p.D, e) && tma_rows(p.g, p.gs, p.D, e) && tma_rows(p.dout, p.ds, p.D, e) &&
           tma_rows(p.dx, p.D, p.D, e) && tma_rows(p.di, p.D, p.D, e) && tma_rows(p.dg, p.D, p.D, e);
}

// Workspace: the scan's, the partial sums, the checkpoints and the forward run's workspace.
struct BwdPlan {
    ScanPlan s;
    float *part_ddt, *part_dA, *checkpoints;
    unsigned char *fwd;
    size_t bytes;
};
BwdPlan bwd_plan(const GlrParams &p, int sms, unsigned char *ws) {
    BwdPlan b;
    size_t at = 0;
    b.s = p.dtype == kFP32 ? scan_plan<BwdShape<float, true>>(p.rows, p.D, ws, &at) : scan_plan<BwdShape<__half, true>>(p.rows, p.D, ws, &at);
    const size_t part = (size_t)(b.s.row_tiles * b.s.width) * sizeof(float);
    const size_t ck = p.checkpoints ? 0 : ((size_t)(b.s.row_tiles * p.D) * sizeof(float) + 15) / 16 * 16;
    b.part_ddt = reinterpret_cast<float *>(ws + at);
    b.part_dA = reinterpret_cast<float *>(ws + at + part);
    b.checkpoints = reinterpret_cast<float *>(ws + at + 2 * part);
    b.fwd = ws + at + 2 * part + ck;
    b.bytes = at + 2 * part + ck + (p.checkpoints ? 0 : glr_fwd_scratch_bytes(states_only(p), sms));
    return b;
}

template <typename E, bool TMA, bool UB>
cudaError_t run(const GlrParams &p, const BwdPlan &b, int sms, cudaStream_t stream) {
    ScanPlan s = b.s;
    using S = BwdShape<E, TMA>;
    using Raw = RawTile<E, S, TMA>;
    ScanMaps<4 * Raw::PHASES> maps{};
    maps.boxed = p.rows >= Raw::PHASES && p.xs >= p.D && p.is >= p.D && p.gs >= p.D && p.ds >= p.D;
    if (maps.boxed &&
        !(encode_maps<Raw>(maps, 0, p.x, p.xs, p.rows, p.D, p.dtype) &&
          encode_maps<Raw>(maps, 1, p.i, p.is, p.rows, p.D, p.dtype) &&
          encode_maps<Raw>(maps, 2, p.g, p.gs, p.rows, p.D, p.dtype) &&
          encode_maps<Raw>(maps, 3, p.dout, p.ds, p.rows, p.D, p.dtype)))
        return cudaErrorUnknown;
    int ctas = 0;
    constexpr int bytes = (int)sizeof(BwdShared<E, TMA>);
    constexpr auto kernel = glr_bwd_scan_kernel<E, TMA, UB>;
    const cudaError_t e = resident_ctas<kernel>(BwdShape<E, TMA>::THREADS, bytes, ctas);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::max(std::min(s.row_tiles * s.blocks, (int64_t)sms * ctas), (int64_t)1);
    GlrParams arg = p;
    float *ddt = b.part_ddt, *dA = b.part_dA;
    void *args[] = {&arg, &s, &maps, &ddt, &dA};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(BwdShape<E, TMA>::THREADS), args,
                                       bytes, stream);
}

}  // namespace

size_t glr_bwd_scratch_bytes(const GlrParams &p, int sms) { return bwd_plan(p, sms, nullptr).bytes; }

cudaError_t launch_glr_bwd(const GlrParams &p0, unsigned char *ws, int sms, cudaStream_t stream) {
    GlrParams p = p0;
    const BwdPlan b = bwd_plan(p, sms, ws);
    cudaError_t e = cudaSuccess;
    if (p.N > 0 && p.D > 0) {
        if (!p.checkpoints) {
            p.checkpoints = b.checkpoints;
            e = launch_glr_fwd(states_only(p), b.fwd, sms, stream);
            if (e != cudaSuccess) return e;
        }
        const bool vec = aligned_rows(p);
        e = with_dtype(p.dtype, [&](auto *tag) {
            using E = std::remove_pointer_t<decltype(tag)>;
            if (vec) return p.unbounded ? run<E, true, true>(p, b, sms, stream) : run<E, true, false>(p, b, sms, stream);
            return p.unbounded ? run<E, false, true>(p, b, sms, stream) : run<E, false, false>(p, b, sms, stream);
        });
        if (e != cudaSuccess) return e;
    }
    if (p.K <= kMaxHead) {
        glr_head_grads_kernel<<<(unsigned)p.H, 1024, 0, stream>>>(p, b.s.row_tiles, b.s.width, b.part_ddt, b.part_dA);
        return cudaGetLastError();
    }
    glr_param_sum_kernel<<<(unsigned)ceil_div(p.D, 32), kSumThreads, 0, stream>>>(p, b.s.row_tiles, b.s.width, b.part_ddt, b.part_dA);
    glr_head_sum_kernel<<<(unsigned)p.H, 128, 0, stream>>>(p, b.s.row_tiles > 0, b.part_dA);
    return cudaGetLastError();
}

}  // namespace kda
