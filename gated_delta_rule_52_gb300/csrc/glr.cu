// Gated linear recurrence, forward: h_t = a_t h_{t-1} + sigma(i_t) x_t per channel, a_t the
// gate's decay (glr_gate.cuh), h in fp32.
//
// Two kernels.  Short fixed-length calls (decode steps) run a thread per (sequence, 4
// channels) over the tokens.  All others run a single pass over tiles of 64 rows
// (glr_scan.cuh): a thread forms a and sigma(i) x of its 8 rows x 4 channels, folds them
// into one affine map, the CTA folds the row groups, hands the tile's map on, takes the
// state that enters the tile, and every thread runs its rows again from its own state with
// a and sigma(i) x still in registers.  Inputs are read once, by copies into shared memory
// that run one tile ahead.
#include <algorithm>

#include "glr_scan.cuh"

namespace kda {
namespace {

using namespace layer;

template <typename E, int V, bool UB>
__global__ void __launch_bounds__(128) glr_fwd_step_kernel(GlrParams p) {
    const int64_t unit = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, per = p.D / V;
    if (unit >= p.N * per) return;
    const int64_t n = unit / per, c = unit % per * V;
    const E *x = static_cast<const E *>(p.x) + n * p.T * p.xs + c;
    const E *i = static_cast<const E *>(p.i) + n * p.T * p.is + c;
    const E *g = static_cast<const E *>(p.g) + n * p.T * p.gs + c;
    E *out = static_cast<E *>(p.out) + n * p.T * p.os + c;
    const float lb2 = p.lower_bound * kLog2e;
    float k0[V], k1[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const GateConst gc = gate_const<UB>(p.A_log[(unsigned)(c + v) / (unsigned)p.K], p.dt_bias[c + v]);
        k0[v] = gc.k0, k1[v] = gc.k1;
        h[v] = p.init ? ld_state(p.init, p.state_type, n * p.D + c + v) : 0.f;
    }
    for (int64_t t = 0; t < p.T; ++t) {
        float xf[V], jf[V], gf[V];
        ld_f<E, V>(x + t * p.xs, xf);
        ld_f<E, V>(i + t * p.is, jf);
        ld_f<E, V>(g + t * p.gs, gf);
        const int64_t row = n * p.T + t;
        if (p.checkpoints && row % kGlrCheckpointRows == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) p.checkpoints[row / kGlrCheckpointRows * p.D + c + v] = h[v];
        }
        float a[V], b[V];
        gate_decay_n<UB, V>(a, gf, k0, k1, lb2);
        sigmoid_n<V>(b, jf);
        mul_n<V>(b, b, xf);
        fma_n<V>(h, a, h, b);
        if (p.out) st_f<E, V>(out + t * p.os, h);
    }
    if (p.fin) {
#pragma unroll
        for (int v = 0; v < V; ++v) st_state(p.fin, p.state_type, n * p.D + c + v, h[v]);
    }
}

// 8 rows by 4 channels per thread.  16 bits: 5 CTAs per SM, 8192 x 8192 bf16 101 us, 5.3 TB/s
// (4 CTAs: 107; 3 CTAs of 256 threads with 4 rows: 131; before the tensor maps, at then 118 us,
// tiles of 32 rows on 7 CTAs 131, and two tiles in flight per CTA, the next one's map handed
// on before the current one's state is taken, on 3 CTAs 163).  What bounds it: the barriers
// between a tile's phases, issue at 57% of the slots.  In 32 bits shared memory holds 4 CTAs,
// 3 of unaligned rows, and the threads have that many more registers: 8192 x 3937 105 us, 114
// with the registers of 5.  Unaligned 16-bit rows: 8192 x 3937 94 us (aligned 3968: 58 us;
// element-wise copies 165 us).
using FwdShape = TileShape<kGlrCheckpointRows, 128, 16, 4>;
template <typename E, bool TMA>
constexpr int kFwdCtas = sizeof(E) == 2 ? 5 : TMA ? 4 : 3;

template <typename E, bool TMA>
struct FwdShared {
    using S = FwdShape;
    RawTile<E, S, TMA> raw[3];                            // x, i, g
    Pack<GateConst, S::V> gates[S::CL];
    Pack<float, S::V> A[S::RG][S::CL], H[S::RG][S::CL];   // maps of the row groups
    Pack<float, S::V> h[S::RG][S::CL];                    // states that enter them
    TileMarks<S::ROWS> marks;
    uint64_t arrived;                                     // of a tile's copies
    int late;
};

template <typename E, bool TMA, bool UB>
__global__ void __launch_bounds__(FwdShape::THREADS, kFwdCtas<E, TMA>)
    glr_fwd_scan_kernel(GlrParams p, ScanPlan s, const __grid_constant__ ScanMaps<3 * RawTile<E, FwdShape, TMA>::PHASES> maps) {
    using namespace sm103;
    using S = FwdShape;
    constexpr int CL = S::CL, V = S::V, L = S::L, CB = S::CB, RG = S::RG;
    extern __shared__ __align__(128) unsigned char smem[];
    FwdShared<E, TMA> &sh = *reinterpret_cast<FwdShared<E, TMA> *>(smem);
    const int tid = threadIdx.x, lane = tid % CL, rg = tid / CL;
    const float lb2 = p.lower_bound * kLog2e;
    const int D = (int)p.D;

    // starts the copies of a tile's inputs
    const auto fetch = [&](const TileWalk &w) {
        if (w.rt >= s.row_tiles) return;
        if (TMA || maps.boxed) {
            fetch_boxes(sh.raw, maps, w.rt * S::ROWS, w.cb * CB, sizeof(sh.gates), &sh.arrived);
        } else if constexpr (!TMA) {
            fetch_elements<E, S, 3>(sh.raw, {p.x, p.i, p.g}, {p.xs, p.is, p.gs}, p.rows, p.D, w.rt * S::ROWS, w.cb * CB,
                                    tid == 0 ? sizeof(sh.gates) : 0, &sh.arrived);
        }
    };
    // and of what the scan's first part has left for the tile; returns its first sequence
    const auto fetch_plan = [&](const TileWalk &w) {
        int first = 0;
        if (w.rt < s.row_tiles) {
            first = s.first_seq[w.rt];
            const GateConst *gates = s.gates + w.cb * CB;
            if (tid == 0) bulk_load(smem_u32(sh.gates), gates, sizeof(sh.gates), smem_u32(&sh.arrived));
        }
        return first;
    };
    const Waits waits{p.err, &sh.late};
    const RowStart<E> starts[3] = {{p.x, p.xs}, {p.i, p.is}, {p.g, p.gs}};

    if (tid == 0) {
        mbar_init(&sh.arrived, TMA || maps.boxed ? 1 : S::THREADS);
        sh.late = 0;
        fence_mbar_init();
    }
    __syncthreads();
    TileWalk w(s);
    fetch(w);
    prepare_scan<UB, false>(p, s);
    fence_proxy_async_global();   // the gates are read by bulk copies
    cooperative_groups::this_grid().sync();
    fence_proxy_async_global();
    int first = fetch_plan(w);
    for (uint32_t parity = 0; w.rt < s.row_tiles; parity ^= 1) {
        const int64_t rt = w.rt, r0 = rt * S::ROWS + rg * L;
        const int block = w.cb * CB, c = block + lane * V;
        const bool marked = mark_tile(p, rt, first, sh.marks);
        const bool plain = !marked && (rt + 1) * S::ROWS <= p.rows;   // every row inside one sequence
        wait_copies(&sh.arrived, parity, waits);

        float a[L][V], b[L][V];
        {
            const ChannelGates<V> gc(sh.gates[lane]);
            const auto raw = [&](int k, int r, float (&f)[V]) {
                unpack<E, V>(TMA ? sh.raw[k].at(rg, r, lane) : pick<E, V>(sh.raw[k].row(rg, r), starts[k][rg * L + r] + lane * V), f);
            };
#pragma unroll
            for (int r = 0; r < L; ++r) {
                float x[V], i[V], g[V];
                raw(0, r, x), raw(1, r, i), raw(2, r, g);
                gate_decay_n<UB, V>(a[r], g, gc.k0, gc.k1, lb2);
                sigmoid_n<V>(b[r], i);
                mul_n<V>(b[r], b[r], x);
            }
        }
        w.next();
        Pack<float, V> mA, mH;
        if (plain) {
#pragma unroll
            for (int v = 0; v < V; ++v) mA.e[v] = a[0][v], mH.e[v] = b[0][v];
#pragma unroll
            for (int r = 1; r < L; ++r) {
                fma_n<V>(mH.e, a[r], mH.e, b[r]);
                mul_n<V>(mA.e, a[r], mA.e);
            }
        } else {
            if (r0 + L > p.rows) {
#pragma unroll
                for (int r = 0; r < L; ++r)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (r0 + r >= p.rows) a[r][v] = 1.f, b[r][v] = 0.f;
            }
            if (marked) {
#pragma unroll
                for (int r = 0; r < L; ++r) {
                    const int n = sh.marks.begins[rg * L + r];
                    if (n < 0) continue;
                    // a row that begins a sequence starts from the initial state instead
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float h0 = p.init && c + v < D ? ld_state(p.init, p.state_type, n * p.D + c + v) : 0.f;
                        b[r][v] = fmaf(a[r][v], h0, b[r][v]);
                        a[r][v] = -0.f;   // depends on nothing before
                        if (r == 0 && rg == 0 && p.checkpoints && c + v < D) p.checkpoints[rt * p.D + c + v] = h0;
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Affine m{a[0][v], b[0][v]};
#pragma unroll
                for (int r = 1; r < L; ++r) m = then(m, Affine{a[r][v], b[r][v]});
                mA.e[v] = m.A, mH.e[v] = m.H;
            }
        }
        sh.A[rg][lane] = mA;
        sh.H[rg][lane] = mH;
        __syncthreads();
        fetch(w);   // the inputs are in registers: the next tile's copies run beside the rest
        first = fetch_plan(w);

        const int64_t group = rt >> s.group_log2;
        const int pos = (int)(rt - (group << s.group_log2)), last = (1 << s.group_log2) - 1;
        const int ch = tid % CB;
        if (tid < CB) {
            // one thread per channel: the tile's map, handed on
            if (pos != last) {
                const GroupMaps<RG, CL, V> maps(sh.A, sh.H, ch);
                Affine t = maps.m[0];
                if (plain) {
#pragma unroll
                    for (int q = 1; q < RG; ++q) t = joined<false>(t, maps.m[q]);
                } else {
#pragma unroll
                    for (int q = 1; q < RG; ++q) t = joined<true>(t, maps.m[q]);
                }
                publish(s.maps + rt * s.width + block + ch, t);
            }
        } else {
            // one thread per channel: the state that enters the tile, from the state after
            // the previous group and the maps of the group's earlier tiles
            const uint32_t *before = s.states + (group - 1) * s.width + block + ch;
            const uint32_t h_bits = group > 0 ? peek(before) : 0;
            const Affine t = join_maps<4>(s.maps + (rt - pos) * s.width + block + ch, s.width, pos, waits);
            float h = apply(t, group > 0 ? __uint_as_float(await(waits, before, h_bits)) : 0.f);
            const GroupMaps<RG, CL, V> maps(sh.A, sh.H, ch);
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                sh.h[q][ch / V].e[ch % V] = h;
                h = plain ? applied<false>(maps.m[q], h) : applied<true>(maps.m[q], h);
            }
            if (pos == last) publish(s.states + group * s.width + block + ch, h);
        }
        __syncthreads();

        const int cols = D - c;
        if (cols > 0) {
            const Pack<float, V> start = sh.h[rg][lane];
            float h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = start.e[v];
            if (p.checkpoints && rg == 0 && !(marked && sh.marks.begins[0] >= 0)) st_cols<float, V, false>(p.checkpoints + rt * p.D + c, h, cols);
            E *out = static_cast<E *>(p.out) + r0 * p.os + c;
            if (plain) {
#pragma unroll
                for (int r = 0; r < L; ++r, out += p.os) {
                    fma_n<V>(h, a[r], h, b[r]);
                    if (p.out) st_cols<E, V, TMA>(out, h, cols);
                }
            } else {
#pragma unroll
                for (int r = 0; r < L; ++r, out += p.os) {
                    if (r0 + r >= p.rows) break;
#pragma unroll
                    for (int v = 0; v < V; ++v) h[v] = apply(Affine{a[r][v], b[r][v]}, h[v]);
                    if (p.out) st_cols<E, V, TMA>(out, h, cols);
                    const int n = marked && p.fin ? sh.marks.ends[rg * L + r] : -1;
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (n >= 0 && v < cols) st_state(p.fin, p.state_type, n * p.D + c + v, h[v]);
                }
            }
        }
    }
}

// Rows of a fixed-length call up to which the step kernel runs.  In a CUDA graph, step and scan:
// 8 x 4 x 128 channels bf16, 16 rows 7.1 and 7.7 us, 24 rows 9.8 and 7.9; 64 sequences of 64 x
// 128, 16 rows 13.3 and 22.6 us.  (With many sequences the step kernel stays ahead for longer,
// 33.9 and 44.7 us at 32 rows; with few, where the call is short, it does not.)
constexpr int64_t kStepMaxT = 16;

bool step_takes(const GlrParams &p) { return !p.cu_seqlens && p.T <= kStepMaxT; }

// Rows that tensor maps take, and 16-byte stores of the step kernel's and the scan's groups.
bool aligned_rows(const GlrParams &p) {
    const size_t e = dtype_bytes(p.dtype);
    return tma_rows(p.x, p.xs, p.D, e) && tma_rows(p.i, p.is, p.D, e) && tma_rows(p.g, p.gs, p.D, e) &&
           (!p.out || tma_rows(p.out, p.os, p.D, e));
}

template <typename E, bool TMA, bool UB>
cudaError_t run(const GlrParams &p, unsigned char *ws, int sms, cudaStream_t stream) {
    if (step_takes(p)) {
        constexpr int V = TMA ? 4 : 1;
        glr_fwd_step_kernel<E, V, UB><<<(unsigned)ceil_div(p.N * (p.D / V), 128), 128, 0, stream>>>(p);
        return cudaGetLastError();
    }
    ScanPlan s = scan_plan<FwdShape>(p.rows, p.D, ws, nullptr);
    using Raw = RawTile<E, FwdShape, TMA>;
    ScanMaps<3 * Raw::PHASES> maps{};
    maps.boxed = p.rows >= Raw::PHASES && p.xs >= p.D && p.is >= p.D && p.gs >= p.D;
    if (maps.boxed &&
        !(encode_maps<Raw>(maps, 0, p.x, p.xs, p.rows, p.D, p.dtype) &&
          encode_maps<Raw>(maps, 1, p.i, p.is, p.rows, p.D, p.dtype) &&
          encode_maps<Raw>(maps, 2, p.g, p.gs, p.rows, p.D, p.dtype)))
        return cudaErrorUnknown;
    constexpr auto kernel = glr_fwd_scan_kernel<E, TMA, UB>;
    constexpr int bytes = (int)sizeof(FwdShared<E, TMA>);
    int ctas = 0;
    const cudaError_t e = resident_ctas<kernel>(FwdShape::THREADS, bytes, ctas);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::max(std::min(s.row_tiles * s.blocks, (int64_t)sms * ctas), (int64_t)1);
    GlrParams arg = p;
    void *args[] = {&arg, &s, &maps};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(FwdShape::THREADS), args, bytes, stream);
}

}  // namespace

size_t glr_fwd_scratch_bytes(const GlrParams &p, int) {
    if (step_takes(p)) return 0;
    size_t bytes = 0;
    scan_plan<FwdShape>(p.rows, p.D, nullptr, &bytes);
    return bytes;
}

cudaError_t launch_glr_fwd(const GlrParams &p, unsigned char *ws, int sms, cudaStream_t stream) {
    return with_dtype(p.dtype, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        if (aligned_rows(p)) return p.unbounded ? run<E, true, true>(p, ws, sms, stream) : run<E, true, false>(p, ws, sms, stream);
        return p.unbounded ? run<E, false, true>(p, ws, sms, stream) : run<E, false, false>(p, ws, sms, stream);
    });
}

}  // namespace kda
