// Host side of the operators around the delta rule declared in include/kda.h (the gated
// linear recurrence, layer norm, the RMS norm, the short convolution, 8-bit tensors and their
// product): argument checks, workspaces from the library's pool, and dispatch to the kernels.
#include <cmath>
#include <cstdint>

#include "../../include/kda.h"
#include "layer.h"

static_assert((int)KDA_DTYPE_BF16 == kda::kBF16 && (int)KDA_DTYPE_FP32 == kda::kFP32 && (int)KDA_DTYPE_FP16 == kda::kFP16 &&
                  (int)KDA_DTYPE_E4M3 == kda::kE4M3 && (int)KDA_DTYPE_E5M2 == kda::kE5M2,
              "element types of include/kda.h");
static_assert(KDA_FP8_BLOCK == kda::kFp8Block, "block of include/kda.h");
static_assert(KDA_GLR_CHECKPOINT_ROWS == kda::kGlrCheckpointRows, "checkpoint spacing of include/kda.h");

namespace {

// Packed rows and channels of one call: both index 32-bit grids and counters.
constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 1;

bool dtype_ok(int dtype) { return dtype == KDA_DTYPE_BF16 || dtype == KDA_DTYPE_FP32 || dtype == KDA_DTYPE_FP16; }
bool fp8_ok(int dtype) { return dtype == KDA_DTYPE_E4M3 || dtype == KDA_DTYPE_E5M2; }
bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t size_of(int dtype) { return dtype == KDA_DTYPE_FP32 ? 4 : 2; }

// Product of two sizes, or -1 where it leaves [0, kMaxExtent].
int64_t extent(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (a == 0 || b == 0) return 0;
    return a > kMaxExtent / b ? -1 : a * b;
}

template <typename Launch>
kda_status with_workspace(size_t bytes, void *stream, Launch &&launch) {
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if (kda::sm_count(sms) != cudaSuccess) return KDA_ERR_CUDA;
    if (bytes == 0) return launch(static_cast<unsigned char *>(nullptr), sms, cs) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return KDA_ERR_CUDA;
    cudaMemPool_t pool = kda::workspace_pool(device);
    if (!pool) return KDA_ERR_CUDA;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, bytes, pool, cs) != cudaSuccess) return KDA_ERR_CUDA;
    kda_status st = launch(static_cast<unsigned char *>(ws), sms, cs) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    if (cudaFreeAsync(ws, cs) != cudaSuccess) st = KDA_ERR_CUDA;
    return st;
}

// Sizes that the recurrence and the convolution share: rows, sequences.
kda_status pack(const int64_t *cu_seqlens, int64_t num_seqs, int64_t B, int64_t T, int64_t &rows, int64_t &N) {
    if (B < 0 || T < 0) return KDA_ERR_SHAPE;
    if (cu_seqlens && (B != 1 || num_seqs < 1)) return KDA_ERR_SHAPE;
    rows = extent(B, T);
    N = cu_seqlens ? num_seqs : B;
    return rows < 0 || N > kMaxExtent ? KDA_ERR_SHAPE : KDA_OK;
}

kda_status fill_glr(const void *x, const void *i, const void *g, int64_t xs, int64_t is, int64_t gs, int dtype,
                    const float *A_log, const float *dt_bias, float lower_bound, int unbounded,
                    const void *init, void *fin, int state_dtype, const int64_t *cu_seqlens, int64_t num_seqs,
                    int64_t B, int64_t T, int64_t H, int64_t K, kda::GlrParams &p) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    kda_status st = pack(cu_seqlens, num_seqs, B, T, p.rows, p.N);
    if (st != KDA_OK) return st;
    p.D = extent(H, K);
    if (p.D < 0 || extent(p.N, p.D) < 0) return KDA_ERR_SHAPE;
    const bool work = p.rows > 0 && p.D > 0;
    if (work && (!x || !i || !g)) return KDA_ERR_NULL;
    if (p.D > 0 && (!A_log || !dt_bias)) return KDA_ERR_NULL;
    if (work && (xs < 0 || is < 0 || gs < 0)) return KDA_ERR_SHAPE;
    if (init || fin) {
        if (state_dtype != KDA_STATE_BF16 && state_dtype != KDA_STATE_FP32) return KDA_ERR_DTYPE;
    } else if (state_dtype != KDA_STATE_NONE && state_dtype != KDA_STATE_BF16 && state_dtype != KDA_STATE_FP32) {
        return KDA_ERR_DTYPE;
    }
    if (!unbounded && !(lower_bound >= -5.0f && lower_bound <= 0.0f)) return KDA_ERR_VALUE;
    const size_t e = size_of(dtype), se = state_dtype == KDA_STATE_BF16 ? 2 : 4;
    if (!aligned_to(x, e) || !aligned_to(i, e) || !aligned_to(g, e) || !aligned_to(A_log, 4) ||
        !aligned_to(dt_bias, 4) || !aligned_to(init, se) || !aligned_to(fin, se) || !aligned_to(cu_seqlens, 8))
        return KDA_ERR_ALIGN;
    p.x = x; p.i = i; p.g = g;
    p.xs = xs; p.is = is; p.gs = gs;
    p.dtype = dtype;
    p.A_log = A_log; p.dt_bias = dt_bias;
    p.lower_bound = lower_bound;
    p.unbounded = unbounded ? 1 : 0;
    p.init = init; p.fin = fin;
    p.state_type = state_dtype;
    p.cu_seqlens = cu_seqlens;
    p.B = B; p.T = T; p.H = H; p.K = K;
    return KDA_OK;
}

kda_status fill_norm(const void *x, int64_t xs, const float *weight, int dtype, int64_t rows, int64_t D,
                     kda::NormParams &p) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (rows < 0 || D < 0 || rows > kMaxExtent || D > kMaxExtent || (rows > 0 && D == 0)) return KDA_ERR_SHAPE;
    if (rows > 0 && !x) return KDA_ERR_NULL;
    if (rows > 0 && xs < 0) return KDA_ERR_SHAPE;
    if (!aligned_to(x, size_of(dtype)) || !aligned_to(weight, 4)) return KDA_ERR_ALIGN;
    p.x = x; p.xs = xs;
    p.weight = weight;
    p.dtype = dtype;
    p.rows = rows; p.D = D;
    return KDA_OK;
}

kda_status fill_rms(const void *x, int64_t xs, const float *weight, int dtype, int64_t rows, int64_t D, kda::RmsParams &p) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (rows < 0 || D < 0 || rows > kMaxExtent || D > kMaxExtent || (rows > 0 && D == 0)) return KDA_ERR_SHAPE;
    if (rows > 0 && !x) return KDA_ERR_NULL;
    if (rows > 0 && xs < 0) return KDA_ERR_SHAPE;
    if (!aligned_to(x, size_of(dtype)) || !aligned_to(weight, 4)) return KDA_ERR_ALIGN;
    p.x = x; p.xs = xs;
    p.weight = weight;
    p.dtype = dtype;
    p.rows = rows; p.D = D;
    return KDA_OK;
}

// Blocks of 128 in n elements.
int64_t fp8_blocks(int64_t n) { return (n + KDA_FP8_BLOCK - 1) / KDA_FP8_BLOCK; }

// Sizes of an 8-bit tensor's call: rows, columns, tiles.
kda_status fill_fp8(int64_t rows, int64_t cols, int dtype, int q_dtype, int tile, kda::QuantParams &p) {
    if (!dtype_ok(dtype) || !fp8_ok(q_dtype)) return KDA_ERR_DTYPE;
    if (rows < 0 || cols < 0 || rows > kMaxExtent || cols > kMaxExtent || extent(fp8_blocks(rows), fp8_blocks(cols)) < 0) return KDA_ERR_SHAPE;
    p.rows = rows; p.cols = cols;
    p.dtype = dtype;
    p.q_dtype = q_dtype;
    p.tile = tile ? 1 : 0;
    return KDA_OK;
}

// An operand of the product; `work`: it is read.
kda_status fill_operand(const void *q, int64_t stride, int q_dtype, const void *scales, int64_t s_stride, int tile, int64_t rows,
                        int64_t K, bool work, kda::Fp8Operand &o) {
    if (!fp8_ok(q_dtype)) return KDA_ERR_DTYPE;
    if (work && (!q || !scales)) return KDA_ERR_NULL;
    const int64_t lines = tile ? fp8_blocks(rows) : rows;
    if (work && ((rows > 1 && stride < K) || (lines > 1 && s_stride < fp8_blocks(K)))) return KDA_ERR_SHAPE;
    if (rows <= 1) stride = (K + 15) / 16 * 16;
    if (lines <= 1) s_stride = 0;
    if (work && (!aligned_to(q, 16) || stride % 16 || !aligned_to(scales, 4) || s_stride % 4)) return KDA_ERR_ALIGN;
    if (work && stride >= int64_t(1) << 40) return KDA_ERR_SHAPE;   // a tensor map's limit
    o.q = q; o.stride = stride; o.rows = rows;
    o.s = static_cast<const uint8_t *>(scales); o.s_stride = s_stride;
    o.tile = tile ? 1 : 0;
    o.dtype = q_dtype;
    return KDA_OK;
}

kda_status fill_conv(const void *x, int64_t xs, const float *weight, const float *bias, int activation, int dtype,
                     const void *init, const int64_t *cu_seqlens, int64_t num_seqs, int64_t B, int64_t T, int64_t D,
                     int64_t W, kda::ConvParams &p) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    if (activation != KDA_ACTIVATION_NONE && activation != KDA_ACTIVATION_SILU) return KDA_ERR_VALUE;
    kda_status st = pack(cu_seqlens, num_seqs, B, T, p.rows, p.N);
    if (st != KDA_OK) return st;
    if (D < 0 || D > kMaxExtent || extent(p.N, D) < 0) return KDA_ERR_SHAPE;
    const bool work = p.rows > 0 && D > 0;
    if (work && !x) return KDA_ERR_NULL;
    if (D > 0 && !weight) return KDA_ERR_NULL;
    if (work && xs < 0) return KDA_ERR_SHAPE;
    const size_t e = size_of(dtype);
    if (!aligned_to(x, e) || !aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(init, e) ||
        !aligned_to(cu_seqlens, 8))
        return KDA_ERR_ALIGN;
    p.x = x; p.xs = xs;
    p.weight = weight; p.bias = bias;
    p.W = (int)W;
    p.silu = activation == KDA_ACTIVATION_SILU;
    p.dtype = dtype;
    p.init = init;
    p.cu_seqlens = cu_seqlens;
    p.B = B; p.T = T; p.D = D;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_glr_fwd(const void *x, const void *i, const void *g, int64_t x_stride, int64_t i_stride,
                       int64_t g_stride, void *out, int64_t out_stride, int dtype, const float *A_log,
                       const float *dt_bias, float lower_bound, int unbounded, const void *initial_state,
                       void *final_state, int state_dtype, const int64_t *cu_seqlens, int64_t num_seqs, int64_t B,
                       int64_t T, int64_t H, int64_t K, float *checkpoints, void *stream) {
    kda::GlrParams p{};
    const kda_status st = fill_glr(x, i, g, x_stride, i_stride, g_stride, dtype, A_log, dt_bias, lower_bound,
                                   unbounded, initial_state, final_state, state_dtype, cu_seqlens, num_seqs, B, T, H,
                                   K, p);
    if (st != KDA_OK) return st;
    if (p.rows > 0 && p.D > 0 && !out) return KDA_ERR_NULL;
    if (p.rows > 1 && p.D > 0 && out_stride < p.D) return KDA_ERR_SHAPE;
    if (!aligned_to(out, size_of(dtype)) || !aligned_to(checkpoints, 4)) return KDA_ERR_ALIGN;
    if (p.N == 0 || p.D == 0) return KDA_OK;
    p.out = out; p.os = out_stride;
    p.checkpoints = checkpoints;
    int sms = 0;
    if (kda::sm_count(sms) != cudaSuccess || kda::device_error_word(p.err) != cudaSuccess) return KDA_ERR_CUDA;
    return with_workspace(kda::glr_fwd_scratch_bytes(p, sms), stream, [&](unsigned char *ws, int n, cudaStream_t cs) {
        return kda::launch_glr_fwd(p, ws, n, cs);
    });
}

kda_status kda_glr_bwd(const void *x, const void *i, const void *g, int64_t x_stride, int64_t i_stride,
                       int64_t g_stride, int dtype, const float *A_log, const float *dt_bias, float lower_bound,
                       int unbounded, const void *initial_state, int state_dtype, const float *checkpoints,
                       const void *dout, int64_t dout_stride, const float *dfinal, const int64_t *cu_seqlens,
                       int64_t num_seqs, int64_t B, int64_t T, int64_t H, int64_t K, void *dx, void *di, void *dg,
                       float *dA_log, float *ddt_bias, float *dinitial_state, void *stream) {
    kda::GlrParams p{};
    const kda_status st = fill_glr(x, i, g, x_stride, i_stride, g_stride, dtype, A_log, dt_bias, lower_bound,
                                   unbounded, initial_state, nullptr, state_dtype, cu_seqlens, num_seqs, B, T, H, K, p);
    if (st != KDA_OK) return st;
    const bool work = p.rows > 0 && p.D > 0;
    if (work && (!dout || !dx || !di || !dg)) return KDA_ERR_NULL;
    if ((H > 0 && !dA_log) || (p.D > 0 && !ddt_bias)) return KDA_ERR_NULL;
    if (work && dout_stride < 0) return KDA_ERR_SHAPE;
    const size_t e = size_of(dtype);
    if (!aligned_to(dout, e) || !aligned_to(dx, e) || !aligned_to(di, e) || !aligned_to(dg, e)) return KDA_ERR_ALIGN;
    if (!aligned_to(checkpoints, 4) || !aligned_to(dfinal, 4) || !aligned_to(dA_log, 4) || !aligned_to(ddt_bias, 4) ||
        !aligned_to(dinitial_state, 4))
        return KDA_ERR_ALIGN;
    if (H == 0) return KDA_OK;
    p.dout = dout; p.ds = dout_stride;
    p.dfinal = dfinal;
    p.checkpoints = const_cast<float *>(checkpoints);
    p.dx = dx; p.di = di; p.dg = dg;
    p.dA_log = dA_log; p.ddt_bias = ddt_bias; p.dinit = dinitial_state;
    int sms = 0;
    if (kda::sm_count(sms) != cudaSuccess || kda::device_error_word(p.err) != cudaSuccess) return KDA_ERR_CUDA;
    return with_workspace(kda::glr_bwd_scratch_bytes(p, sms), stream, [&](unsigned char *ws, int n, cudaStream_t cs) {
        return kda::launch_glr_bwd(p, ws, n, cs);
    });
}

kda_status kda_layer_norm_fwd(const void *x, int64_t x_stride, const float *weight, const float *bias, float eps,
                              void *out, int64_t out_stride, float *mean, float *rstd, int dtype, int64_t rows,
                              int64_t D, void *stream) {
    kda::NormParams p{};
    const kda_status st = fill_norm(x, x_stride, weight, dtype, rows, D, p);
    if (st != KDA_OK) return st;
    if (rows > 0 && !out) return KDA_ERR_NULL;
    if (rows > 1 && out_stride < D) return KDA_ERR_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return KDA_ERR_VALUE;
    if (!aligned_to(out, size_of(dtype)) || !aligned_to(bias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return KDA_ERR_ALIGN;
    if (rows == 0) return KDA_OK;
    p.bias = bias;
    p.eps = eps;
    p.out = out; p.os = out_stride;
    p.mean = mean; p.rstd = rstd;
    return with_workspace(0, stream, [&](unsigned char *, int n, cudaStream_t cs) { return kda::launch_norm_fwd(p, n, cs); });
}

kda_status kda_layer_norm_bwd(const void *dout, int64_t dout_stride, const void *x, int64_t x_stride,
                              const float *weight, const float *mean, const float *rstd, void *dx, float *dweight,
                              float *dbias, int dtype, int64_t rows, int64_t D, void *stream) {
    kda::NormParams p{};
    const kda_status st = fill_norm(x, x_stride, weight, dtype, rows, D, p);
    if (st != KDA_OK) return st;
    if (rows > 0 && (!dout || !mean || !rstd || !dx)) return KDA_ERR_NULL;
    if (rows > 0 && dout_stride < 0) return KDA_ERR_SHAPE;
    const size_t e = size_of(dtype);
    if (!aligned_to(dout, e) || !aligned_to(dx, e) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
        return KDA_ERR_ALIGN;
    if (D == 0 || (rows == 0 && !dweight && !dbias)) return KDA_OK;
    p.dout = dout; p.ds = dout_stride;
    p.mean = const_cast<float *>(mean); p.rstd = const_cast<float *>(rstd);
    p.dx = dx;
    p.dweight = dweight; p.dbias = dbias;
    int sms = 0;
    if (kda::sm_count(sms) != cudaSuccess) return KDA_ERR_CUDA;
    return with_workspace(kda::norm_bwd_scratch_bytes(p, sms), stream, [&](unsigned char *ws, int n, cudaStream_t cs) {
        return kda::launch_norm_bwd(p, ws, n, cs);
    });
}

kda_status kda_short_conv_fwd(const void *x, int64_t x_stride, const float *weight, const float *bias, int activation,
                              void *out, int64_t out_stride, int dtype, const void *initial_state, void *final_state,
                              const int64_t *cu_seqlens, int64_t num_seqs, int64_t B, int64_t T, int64_t D, int64_t W,
                              void *stream) {
    kda::ConvParams p{};
    const kda_status st = fill_conv(x, x_stride, weight, bias, activation, dtype, initial_state, cu_seqlens, num_seqs,
                                    B, T, D, W, p);
    if (st != KDA_OK) return st;
    const bool work = p.rows > 0 && D > 0;
    if (work && !out) return KDA_ERR_NULL;
    if (p.rows > 1 && D > 0 && out_stride < D) return KDA_ERR_SHAPE;
    if (!aligned_to(out, size_of(dtype)) || !aligned_to(final_state, size_of(dtype))) return KDA_ERR_ALIGN;
    if (p.N == 0 || D == 0) return KDA_OK;
    p.out = out; p.os = out_stride;
    p.fin = final_state;
    return with_workspace(0, stream, [&](unsigned char *, int n, cudaStream_t cs) { return kda::launch_conv_fwd(p, n, cs); });
}

kda_status kda_short_conv_bwd(const void *x, int64_t x_stride, const float *weight, const float *bias, int activation,
                              int dtype, const void *initial_state, const void *dout, int64_t dout_stride,
                              const float *dfinal, const int64_t *cu_seqlens, int64_t num_seqs, int64_t B, int64_t T,
                              int64_t D, int64_t W, void *dx, float *dweight, float *dbias, float *dinitial_state,
                              void *stream) {
    kda::ConvParams p{};
    const kda_status st = fill_conv(x, x_stride, weight, bias, activation, dtype, initial_state, cu_seqlens, num_seqs,
                                    B, T, D, W, p);
    if (st != KDA_OK) return st;
    const bool work = p.rows > 0 && D > 0;
    if (work && (!dout || !dx)) return KDA_ERR_NULL;
    if (D > 0 && !dweight) return KDA_ERR_NULL;
    if (work && dout_stride < 0) return KDA_ERR_SHAPE;
    const size_t e = size_of(dtype);
    if (!aligned_to(dout, e) || !aligned_to(dx, e) || !aligned_to(dfinal, 4) || !aligned_to(dweight, 4) ||
        !aligned_to(dbias, 4) || !aligned_to(dinitial_state, 4))
        return KDA_ERR_ALIGN;
    if (D == 0) return KDA_OK;
    p.dout = dout; p.ds = dout_stride;
    p.dfinal = dfinal;
    p.dx = dx;
    p.dweight = dweight; p.dbias = dbias; p.dinit = dinitial_state;
    int sms = 0;
    if (kda::sm_count(sms) != cudaSuccess) return KDA_ERR_CUDA;
    return with_workspace(kda::conv_bwd_scratch_bytes(p, sms), stream, [&](unsigned char *ws, int n, cudaStream_t cs) {
        return kda::launch_conv_bwd(p, ws, n, cs);
    });
}

kda_status kda_rms_norm_fwd(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, const float *weight,
                            float eps, void *out, int64_t out_stride, int out_dtype, void *scales, int64_t scales_stride,
                            void *residual_out, int64_t residual_out_stride, float *rstd, int dtype, int64_t rows, int64_t D,
                            void *stream) {
    kda::RmsParams p{};
    const kda_status st = fill_rms(x, x_stride, weight, dtype, rows, D, p);
    if (st != KDA_OK) return st;
    const bool small = fp8_ok(out_dtype);
    if (!small && out_dtype != dtype) return KDA_ERR_DTYPE;
    if (rows > 0 && (!out || (small && !scales))) return KDA_ERR_NULL;
    if (residual_out && !residual) return KDA_ERR_NULL;
    if (rows > 0 && residual && residual_stride < 0) return KDA_ERR_SHAPE;
    if (rows > 1 && (out_stride < D || (residual_out && residual_out_stride < D) || (small && scales_stride < fp8_blocks(D))))
        return KDA_ERR_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return KDA_ERR_VALUE;
    const size_t e = size_of(dtype);
    if ((!small && !aligned_to(out, e)) || !aligned_to(residual, e) || !aligned_to(residual_out, e) || !aligned_to(rstd, 4))
        return KDA_ERR_ALIGN;
    if (rows == 0) return KDA_OK;
    p.res = residual; p.rs = residual_stride;
    p.eps = eps;
    p.out = out; p.os = out_stride; p.out_dtype = out_dtype;
    p.scales = static_cast<uint8_t *>(scales); p.ss = scales_stride;
    p.res_out = residual_out; p.ros = residual_out_stride;
    p.rstd = rstd;
    return with_workspace(0, stream, [&](unsigned char *, int n, cudaStream_t cs) { return kda::launch_rms_fwd(p, n, cs); });
}

kda_status kda_rms_norm_bwd(const void *dout, int64_t dout_stride, const void *x, int64_t x_stride, const float *weight,
                            const float *rstd, const void *dresidual, int64_t dresidual_stride, void *dx, float *dweight,
                            int dtype, int64_t rows, int64_t D, void *stream) {
    kda::RmsParams p{};
    const kda_status st = fill_rms(x, x_stride, weight, dtype, rows, D, p);
    if (st != KDA_OK) return st;
    if (rows > 0 && (!dout || !rstd || !dx)) return KDA_ERR_NULL;
    if (rows > 0 && (dout_stride < 0 || (dresidual && dresidual_stride < 0))) return KDA_ERR_SHAPE;
    const size_t e = size_of(dtype);
    if (!aligned_to(dout, e) || !aligned_to(dresidual, e) || !aligned_to(dx, e) || !aligned_to(rstd, 4) || !aligned_to(dweight, 4))
        return KDA_ERR_ALIGN;
    if (D == 0 || (rows == 0 && !dweight)) return KDA_OK;
    p.dout = dout; p.ds = dout_stride;
    p.dres = dresidual; p.drs = dresidual_stride;
    p.rstd = const_cast<float *>(rstd);
    p.dx = dx;
    p.dweight = dweight;
    int sms = 0;
    if (kda::sm_count(sms) != cudaSuccess) return KDA_ERR_CUDA;
    return with_workspace(kda::rms_bwd_scratch_bytes(p, sms), stream, [&](unsigned char *ws, int n, cudaStream_t cs) {
        return kda::launch_rms_bwd(p, ws, n, cs);
    });
}

kda_status kda_fp8_quantize(const void *x, int64_t x_stride, int dtype, void *q, int64_t q_stride, void *scales,
                            int64_t scales_stride, void *qt, int64_t qt_stride, void *scales_t, int64_t scales_t_stride,
                            int q_dtype, int tile, int64_t rows, int64_t cols, void *stream) {
    kda::QuantParams p{};
    const kda_status st = fill_fp8(rows, cols, dtype, q_dtype, tile, p);
    if (st != KDA_OK) return st;
    if ((q && !scales) || (qt && !scales_t) || (!q && scales) || (!qt && scales_t)) return KDA_ERR_NULL;
    const bool work = rows > 0 && cols > 0;
    if (work && (!x || (!q && !qt))) return KDA_ERR_NULL;
    if (work && x_stride < 0) return KDA_ERR_SHAPE;
    const int64_t br = fp8_blocks(rows), bc = fp8_blocks(cols);
    if (work && q && ((rows > 1 && q_stride < cols) || ((tile ? br : rows) > 1 && scales_stride < bc))) return KDA_ERR_SHAPE;
    if (work && qt && ((cols > 1 && qt_stride < rows) || ((tile ? bc : cols) > 1 && scales_t_stride < br))) return KDA_ERR_SHAPE;
    if (!aligned_to(x, size_of(dtype))) return KDA_ERR_ALIGN;
    if (!work) return KDA_OK;
    p.x = x; p.xs = x_stride;
    p.q = q; p.qs = q_stride;
    p.qt = qt; p.qts = qt_stride;
    p.s = static_cast<uint8_t *>(scales); p.ss = scales_stride;
    p.st = static_cast<uint8_t *>(scales_t); p.sts = scales_t_stride;
    return with_workspace(0, stream, [&](unsigned char *, int n, cudaStream_t cs) { return kda::launch_quantize(p, n, cs); });
}

kda_status kda_fp8_dequantize(const void *q, int64_t q_stride, int q_dtype, const void *scales, int64_t scales_stride, int tile,
                              void *out, int64_t out_stride, int dtype, int64_t rows, int64_t cols, void *stream) {
    kda::QuantParams p{};
    const kda_status st = fill_fp8(rows, cols, dtype, q_dtype, tile, p);
    if (st != KDA_OK) return st;
    const bool work = rows > 0 && cols > 0;
    if (work && (!q || !scales || !out)) return KDA_ERR_NULL;
    if (work && (q_stride < 0 || scales_stride < 0 || (rows > 1 && out_stride < cols))) return KDA_ERR_SHAPE;
    if (!aligned_to(out, size_of(dtype))) return KDA_ERR_ALIGN;
    if (!work) return KDA_OK;
    p.x = out; p.xs = out_stride;
    p.q = const_cast<void *>(q); p.qs = q_stride;
    p.s = static_cast<uint8_t *>(const_cast<void *>(scales)); p.ss = scales_stride;
    return with_workspace(0, stream, [&](unsigned char *, int n, cudaStream_t cs) { return kda::launch_dequantize(p, n, cs); });
}

kda_status kda_fp8_matmul(const void *a, int64_t a_stride, int a_dtype, const void *a_scales, int64_t a_scales_stride, int a_tile,
                          const void *b, int64_t b_stride, int b_dtype, const void *b_scales, int64_t b_scales_stride, int b_tile,
                          void *out, int64_t out_stride, const void *add, int64_t add_stride, int dtype, int64_t M, int64_t N,
                          int64_t K, void *stream) {
    kda::MatmulParams p{};
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (M < 0 || N < 0 || K < 0 || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return KDA_ERR_SHAPE;
    const bool some = M > 0 && N > 0, work = some && K > 0;
    kda_status st = fill_operand(a, a_stride, a_dtype, a_scales, a_scales_stride, a_tile, M, K, work, p.a);
    if (st == KDA_OK) st = fill_operand(b, b_stride, b_dtype, b_scales, b_scales_stride, b_tile, N, K, work, p.b);
    if (st != KDA_OK) return st;
    if (some && !out) return KDA_ERR_NULL;
    if ((some && M > 1 && out_stride < N) || (add && add_stride < 0)) return KDA_ERR_SHAPE;
    // 128 x 16 is the smallest tile
    if (extent(fp8_blocks(N) * 8, (M + 15) / 16) < 0) return KDA_ERR_SHAPE;
    if (!aligned_to(out, size_of(dtype)) || !aligned_to(add, size_of(dtype))) return KDA_ERR_ALIGN;
    if (!some) return KDA_OK;
    p.out = out; p.os = out_stride;
    p.add = add; p.as = add_stride;
    p.dtype = dtype;
    p.K = K;
    if (kda::device_error_word(p.err) != cudaSuccess) return KDA_ERR_CUDA;
    return with_workspace(0, stream, [&](unsigned char *, int n, cudaStream_t cs) { return kda::launch_matmul(p, n, cs); });
}

}  // extern "C"
