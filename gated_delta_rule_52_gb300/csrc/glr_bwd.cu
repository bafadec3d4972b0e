// Gated linear recurrence, backward.  With e_t the gradient of h_t and f_t = a_t e_t what
// passes on to h_{t-1},
//   e_t = dout_t + f_{t+1}   (of a sequence's last token also + dfinal)
//   f_t = a_t f_{t+1} + a_t dout_t
//   dx = e s, di = e x s (1 - s), s = sigma(i);   dl = f_t h_{t-1}, the gradient of gk_t;
//   dg = dl d gk/dg, ddt_bias = sum dg, dA_log = sum dl d gk/dA_log, dinit = f_first.
//
// One pass over tiles of 64 rows from the last to the first (glr_scan.cuh).  h_{t-1} is
// recomputed in fp32: a tile's rows are those of one checkpoint, so the forward states need
// no other tile.  A thread forms the decays of its 16 elements and folds them forward (from
// the checkpoint) and backward (into the map that the tile hands on); with the states that
// enter its rows from both sides it then forms the gradients, the inputs still in shared
// memory and three values per element in registers.  Inputs are read and gradients written
// once.  Parameter gradients leave a tile as one partial sum per channel.
#include <algorithm>

#include "glr_scan.cuh"

namespace kda {
namespace {

using namespace layer;

// 16 elements per thread: 4 rows by 4 channels in 16 bits, 8 by 2 in 32 bits (the raw
// inputs of two tiles in shared memory allow 2 and 3 CTAs per SM), 16 by 1 where rows are
// not aligned.
template <typename E, int V> using BwdShape = TileShape<V == 4 ? 256 : 128, V == 1 ? 32 : 16, V>;

template <typename E, int V>
struct BwdShared {
    using S = BwdShape<E, V>;
    Pack<E, V> raw[2][4][S::L][S::THREADS];                  // x, i, g, dout
    Pack<GateConst, V> gates[2][S::THREADS];
    Pack<float, V> A[S::RG][S::CL], H[S::RG][S::CL];         // forward maps of the row groups
    Pack<float, V> B[S::RG][S::CL], F[S::RG][S::CL];         // backward maps
    Pack<float, V> h[S::RG][S::CL], f[S::RG][S::CL];         // states that enter them
    Pack<float, V> sum_ddt[S::RG][S::CL], sum_dA[S::RG][S::CL];
    TileMarks marks;
};

template <typename E, int V, bool UB>
__global__ void __launch_bounds__(BwdShape<E, V>::THREADS, V == 4 ? 2 : 3)
    glr_bwd_scan_kernel(GlrParams p, ScanPlan s, float *part_ddt, float *part_dA) {
    using namespace sm103;
    using S = BwdShape<E, V>;
    constexpr int CL = S::CL, L = S::L, CB = S::CB, RG = S::RG;
    static_assert(S::THREADS >= 3 * CB && L * V == 16, "roles");
    extern __shared__ __align__(16) unsigned char smem[];
    BwdShared<E, V> &sh = *reinterpret_cast<BwdShared<E, V> *>(smem);
    const int tid = threadIdx.x, lane = tid % CL, rg = tid / CL;
    const int role = tid / CB, ch = tid % CB;
    const float lb2 = p.lower_bound * kLog2e;
    float checkpoint = 0.f;   // of role 2's channel, fetched with the tile

    // tile number w.rt counts from the last row tile
    auto fetch = [&](const TileWalk &w, int stage) {
        int first = 0;
        if (w.rt < s.row_tiles) {
            const int64_t rt = s.row_tiles - 1 - w.rt, r0 = rt * kTileRows + rg * L;
            const int c = w.cb * CB + lane * V;
            first = s.first_seq[rt];
            const float *gate = reinterpret_cast<const float *>(s.gates + c);
            copy_async<float, V == 4 ? 4 : 2 * V>(&sh.gates[stage][tid], gate);
            if (V == 4) copy_async<float, 4>(&sh.gates[stage][tid].e[V / 2], gate + 4);
            if (role == 2 && w.cb * CB + ch < p.D) checkpoint = p.checkpoints[rt * p.D + w.cb * CB + ch];
            if (c < p.D) {
                const int left = (int)min(p.rows - r0, (int64_t)L);
                const auto copy = [&](int k, const void *src, int64_t stride) {
                    copy_rows<E, V, L, S::THREADS>(&sh.raw[stage][k][0][tid], static_cast<const E *>(src) + r0 * stride + c,
                                                   stride, left);
                };
                copy(0, p.x, p.xs);
                copy(1, p.i, p.is);
                copy(2, p.g, p.gs);
                copy(3, p.dout, p.ds);
            }
        }
        copies_commit();
        return first;
    };

    TileWalk w(s);
    int next_first = fetch(w, 0);
    for (int stage = 0; w.rt < s.row_tiles; stage ^= 1) {
        const int64_t walk = w.rt, rt = s.row_tiles - 1 - walk, r0 = rt * kTileRows + rg * L;
        const int c = w.cb * CB + lane * V, block = w.cb * CB, first = next_first;
        const float h_tile = checkpoint;
        w.next();
        next_first = fetch(w, stage ^ 1);
        const bool marked = mark_tile(p, rt, first, sh.marks);
        copies_wait<1>();   // this thread's own copies: no barrier needed

        const int left = c < p.D ? (int)min(p.rows - r0, (int64_t)L) : 0;   // rows of this thread that exist
        const ChunkGates<V> gc(sh.gates[stage][tid]);
        const auto raw = [&](int k) { return &sh.raw[stage][k][0][tid]; };
        constexpr int n = kGateWidth<V>;
        float a[L][V], mg[L][V], mi[L][V];   // kept for the second half
        Pack<float, V> mA, mH, mB, mF;
#pragma unroll
        for (int v = 0; v < V; ++v) mA.e[v] = mB.e[v] = 1.f, mH.e[v] = mF.e[v] = 0.f;
#pragma unroll
        for (int e = 0; e < L * V; e += n) {
            float x[n], i[n], g[n], d[n], ac[n], s[n], mgc[n], mic[n];
            ld_chunk<E, V, S::THREADS>(raw(0), e, x);
            ld_chunk<E, V, S::THREADS>(raw(1), e, i);
            ld_chunk<E, V, S::THREADS>(raw(2), e, g);
            ld_chunk<E, V, S::THREADS>(raw(3), e, d);
            token_gates_n<UB, n>(ac, s, mgc, mic, g, i, gc.k0, gc.k1, lb2);
            mul_n<n>(s, s, x);
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const int r = (e + j) / V, v = (e + j) % V;
                a[r][v] = ac[j], mg[r][v] = mgc[j], mi[r][v] = mic[j];
            }
            if (!marked && left == L) {
                // forward: after the rows before; backward: f = a_0 (dout_0 + a_1 (dout_1 + ...))
#pragma unroll
                for (int j = 0; j < n; j += V) {
                    const auto &ar = reinterpret_cast<const float (&)[V]>(ac[j]);
                    fma_n<V>(mH.e, ar, mH.e, reinterpret_cast<const float (&)[V]>(s[j]));
                    mul_n<V>(mA.e, ar, mA.e);
                    fma_n<V>(mF.e, mA.e, reinterpret_cast<const float (&)[V]>(d[j]), mF.e);
                }
            } else {
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const int r = (e + j) / V, v = (e + j) % V;
                    if (r >= left) continue;
                    const int begins = marked ? sh.marks.begins[rg * L + r] : -1, ends = marked ? sh.marks.ends[rg * L + r] : -1;
                    if (begins >= 0) {
                        const float h0 = p.init ? ld_state(p.init, p.state_type, begins * p.D + c + v) : 0.f;
                        mA.e[v] = -0.f, mH.e[v] = fmaf(ac[j], h0, s[j]);
                    } else {
                        mH.e[v] = fmaf(ac[j], mH.e[v], s[j]);
                        mA.e[v] *= ac[j];
                    }
                    // backward map of rows 0 .. r: the earlier rows' map after this row's
                    const float dt = ends >= 0 && p.dfinal ? d[j] + p.dfinal[ends * p.D + c + v] : d[j];
                    const Affine m = then(Affine{ends >= 0 ? -0.f : ac[j], ac[j] * dt}, Affine{mB.e[v], mF.e[v]});
                    mB.e[v] = m.A, mF.e[v] = m.H;
                }
            }
        }
        if (!marked && left == L) mB = mA;
        sh.A[rg][lane] = mA;
        sh.H[rg][lane] = mH;
        sh.B[rg][lane] = mB;
        sh.F[rg][lane] = mF;
        __syncthreads();

        const int64_t group = walk >> s.group_log2;
        const int pos = (int)(walk - (group << s.group_log2)), last = (1 << s.group_log2) - 1;
        const auto back = [&](int q) { return Affine{sh.B[q][ch / V].e[ch % V], sh.F[q][ch / V].e[ch % V]}; };
        if (role == 0) {
            // the tile's backward map, handed on
            if (pos != last) {
                Affine t = back(RG - 1);
#pragma unroll
                for (int q = RG - 2; q >= 0; --q) t = then(t, back(q));
                publish(s.maps + walk * s.width + block + ch, t);
            }
        } else if (role == 1) {
            // what enters the tile and its row groups from behind
            const uint32_t *before = s.states + (group - 1) * s.width + block + ch;
            const uint32_t f_bits = group > 0 ? peek(before) : 0;
            const Affine t = join_maps(s.maps + (walk - pos) * s.width + block + ch, s.width, pos, p.err);
            float f = apply(t, group > 0 ? __uint_as_float(await(before, f_bits, p.err)) : 0.f);
#pragma unroll
            for (int q = RG - 1; q >= 0; --q) {
                sh.f[q][ch / V].e[ch % V] = f;
                f = apply(back(q), f);
            }
            if (pos == last) publish(s.states + group * s.width + block + ch, f);
        } else if (role == 2) {
            // the forward states that enter the row groups
            float h = h_tile;
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                sh.h[q][ch / V].e[ch % V] = h;
                h = apply(Affine{sh.A[q][ch / V].e[ch % V], sh.H[q][ch / V].e[ch % V]}, h);
            }
        }
        __syncthreads();

        Pack<float, V> ddt, dA;
#pragma unroll
        for (int v = 0; v < V; ++v) ddt.e[v] = dA.e[v] = 0.f;
        if (left > 0) {
            float start[L][V], h[V], f[V];   // the states that the rows start from
            const Pack<float, V> h_in = sh.h[rg][lane], f_in = sh.f[rg][lane];
            const auto &k0 = reinterpret_cast<const float (&)[V]>(gc.k0), &k1 = reinterpret_cast<const float (&)[V]>(gc.k1);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = h_in.e[v], f[v] = f_in.e[v];
#pragma unroll
            for (int r = 0; r < L; ++r) {
                if (marked && r < left && sh.marks.begins[rg * L + r] >= 0) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        h[v] = p.init ? ld_state(p.init, p.state_type, sh.marks.begins[rg * L + r] * p.D + c + v) : 0.f;
                }
#pragma unroll
                for (int v = 0; v < V; ++v) start[r][v] = h[v];
                if (r == L - 1) break;
                float x[V], i[V], s[V];
                unpack<E, V>(*(raw(0) + r * S::THREADS), x);
                unpack<E, V>(*(raw(1) + r * S::THREADS), i);
                fma_n<V>(s, mi[r], -1.f, 1.f);
#pragma unroll
                for (int v = 0; v < V; ++v) s[v] = i[v] >= 0.f ? s[v] : mi[r][v];
                mul_n<V>(s, s, x);
                fma_n<V>(h, a[r], h, s);
            }
            const int64_t row_at = (r0 + L - 1) * p.D + c;
            E *dx = static_cast<E *>(p.dx) + row_at, *di = static_cast<E *>(p.di) + row_at, *dg = static_cast<E *>(p.dg) + row_at;
#pragma unroll
            for (int r = L - 1; r >= 0; --r, dx -= p.D, di -= p.D, dg -= p.D) {
                if (r >= left) continue;
                if (marked && sh.marks.ends[rg * L + r] >= 0) {
#pragma unroll
                    for (int v = 0; v < V; ++v) f[v] = p.dfinal ? p.dfinal[sh.marks.ends[rg * L + r] * p.D + c + v] : 0.f;
                }
                float x[V], i[V], g[V], grad[V], gm[V], go[V], o[V], slope[V], rate[V];
                unpack<E, V>(*(raw(0) + r * S::THREADS), x);
                unpack<E, V>(*(raw(1) + r * S::THREADS), i);
                unpack<E, V>(*(raw(2) + r * S::THREADS), g);
                unpack<E, V>(*(raw(3) + r * S::THREADS), grad);
                add_n<V>(grad, grad, f);
                mul_n<V>(f, a[r], grad);
                if (marked && p.dinit && sh.marks.begins[rg * L + r] >= 0) {
#pragma unroll
                    for (int v = 0; v < V; ++v) p.dinit[sh.marks.begins[rg * L + r] * p.D + c + v] = f[v];
                }
                fma_n<V>(o, mi[r], -1.f, 1.f);
                mul_n<V>(gm, grad, mi[r]);
                mul_n<V>(go, grad, o);
                float out[V];
#pragma unroll
                for (int v = 0; v < V; ++v) out[v] = i[v] >= 0.f ? go[v] : gm[v];
                st_f<E, V>(dx, out);
                mul_n<V>(out, gm, o);
                mul_n<V>(out, out, x);
                st_f<E, V>(di, out);
                gate_slopes_n<UB, V>(slope, rate, g, mg[r], k0, k1, p.lower_bound);
                mul_n<V>(o, f, start[r]);        // the gradient of gk
                mul_n<V>(out, o, slope);
                st_f<E, V>(dg, out);
                add_n<V>(ddt.e, ddt.e, out);
                fma_n<V>(dA.e, o, rate, dA.e);
            }
        }
        sh.sum_ddt[rg][lane] = ddt;
        sh.sum_dA[rg][lane] = dA;
        __syncthreads();
        if (role < 2) {
            const auto &sum = role == 0 ? sh.sum_ddt : sh.sum_dA;
            float t = 0.f;
#pragma unroll
            for (int q = 0; q < RG; ++q) t += sum[q][ch / V].e[ch % V];
            (role == 0 ? part_ddt : part_dA)[rt * s.width + block + ch] = t;
        }
    }
    copies_wait<0>();
}

// Sums the tiles' partial parameter gradients [parts, width] over the tiles, 32 channels
// per CTA: ddt_bias, and in part_dA's first row dA_log's sums per channel.
__global__ void __launch_bounds__(1024) glr_param_sum_kernel(GlrParams p, int64_t parts, int64_t width, const float *part_ddt,
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

// V channels per thread where every row of the inputs and gradients allows it.
bool vector_rows(const GlrParams &p) {
    const size_t V = p.dtype == kFP32 ? 2 : 4, n = V * dtype_bytes(p.dtype);
    const void *ptrs[] = {p.x, p.i, p.g, p.dout, p.dx, p.di, p.dg};
    for (const void *q : ptrs)
        if (reinterpret_cast<uintptr_t>(q) % n) return false;
    return p.D % V == 0 && p.xs % V == 0 && p.is % V == 0 && p.gs % V == 0 && p.ds % V == 0;
}
int block_channels(const GlrParams &p) { return vector_rows(p) && p.dtype != kFP32 ? 64 : 32; }

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
    b.s = scan_plan(p.rows, p.D, block_channels(p), ws, &at);
    const size_t part = (size_t)(b.s.row_tiles * b.s.width) * sizeof(float);
    const size_t ck = p.checkpoints ? 0 : ((size_t)(b.s.row_tiles * p.D) * sizeof(float) + 15) / 16 * 16;
    b.part_ddt = reinterpret_cast<float *>(ws + at);
    b.part_dA = reinterpret_cast<float *>(ws + at + part);
    b.checkpoints = reinterpret_cast<float *>(ws + at + 2 * part);
    b.fwd = ws + at + 2 * part + ck;
    b.bytes = at + 2 * part + ck + (p.checkpoints ? 0 : glr_fwd_scratch_bytes(states_only(p), sms));
    return b;
}

template <typename E, int V, bool UB>
cudaError_t run(const GlrParams &p, const BwdPlan &b, int sms, cudaStream_t stream) {
    ScanPlan s = b.s;
    const int64_t fill = s.row_tiles * s.width / 2 + s.width;
    glr_prepare_kernel<UB, true><<<(unsigned)std::min(ceil_div(fill, 256), (int64_t)sms * 4), 256, 0, stream>>>(p, s);
    if (s.row_tiles == 0) return cudaGetLastError();
    int ctas = 0;
    constexpr int bytes = (int)sizeof(BwdShared<E, V>);
    constexpr auto kernel = glr_bwd_scan_kernel<E, V, UB>;
    const cudaError_t e = resident_ctas<kernel>(BwdShape<E, V>::THREADS, bytes, ctas);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::min(s.row_tiles * s.blocks, (int64_t)sms * ctas);
    GlrParams arg = p;
    float *ddt = b.part_ddt, *dA = b.part_dA;
    void *args[] = {&arg, &s, &ddt, &dA};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(BwdShape<E, V>::THREADS), args,
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
        const bool vec = vector_rows(p);
        e = with_dtype(p.dtype, [&](auto *tag) {
            using E = std::remove_pointer_t<decltype(tag)>;
            constexpr int V = sizeof(E) == 4 ? 2 : 4;
            if (vec) return p.unbounded ? run<E, V, true>(p, b, sms, stream) : run<E, V, false>(p, b, sms, stream);
            return p.unbounded ? run<E, 1, true>(p, b, sms, stream) : run<E, 1, false>(p, b, sms, stream);
        });
        if (e != cudaSuccess) return e;
    }
    if (p.D > 0)
        glr_param_sum_kernel<<<(unsigned)ceil_div(p.D, 32), 1024, 0, stream>>>(p, b.s.row_tiles, b.s.width, b.part_ddt, b.part_dA);
    glr_head_sum_kernel<<<(unsigned)p.H, 128, 0, stream>>>(p, b.s.row_tiles > 0, b.part_dA);
    return cudaGetLastError();
}

}  // namespace kda
