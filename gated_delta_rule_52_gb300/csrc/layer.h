// Launch parameters shared by the host entry points (layer_api.cu) and the kernels of the
// operators around the delta rule: the gated linear recurrence (glr*.cu), layer norm
// (layer_norm.cu), the RMS norm (rms_norm.cu), the short causal convolution (short_conv.cu),
// and quantisation to 8 bits and the product of such tensors (fp8_quant.cu, fp8_mm.cu).  Not
// part of the public ABI (that is include/kda.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kda_internal.h"

namespace kda {

// Element types of the operators' tensors (KDA_DTYPE_* of include/kda.h).
enum DType : int { kBF16 = 1, kFP32 = 2, kFP16 = 3, kE4M3 = 4, kE5M2 = 5 };

// The library's memory pool of a device and the device error word (kda_api.cu).
cudaMemPool_t workspace_pool(int device);
cudaError_t device_error_word(int *&err);

// ------------------------------------------------------- gated linear recurrence
constexpr int kGlrCheckpointRows = 64;

// Tensors are [rows, D] with D = H*K contiguous channels per packed row and the given row
// strides (elements); states are [N, D].  Sequence n is rows [n*T, (n+1)*T), or
// [cu_seqlens[n], cu_seqlens[n+1]).
struct GlrParams {
    const void *x, *i, *g;
    int64_t xs, is, gs;            // row strides of x, i, g
    void *out;                     // may be null: outputs not written
    int64_t os;
    int dtype;
    const float *A_log, *dt_bias;
    float lower_bound;
    int unbounded;
    const void *init;              // null = zero state
    void *fin;                     // null = not written
    int state_type;
    const int64_t *cu_seqlens;
    int64_t N, B, T, H, K, D, rows;
    float *checkpoints;            // fp32 [ceil(rows/64), D]; written forward, read backward
    int *err;
    // backward only
    const void *dout;
    int64_t ds;
    const float *dfinal;
    void *dx, *di, *dg;            // [rows, D] contiguous, dtype
    float *dA_log, *ddt_bias, *dinit;
};
size_t glr_fwd_scratch_bytes(const GlrParams &p, int sms);
size_t glr_bwd_scratch_bytes(const GlrParams &p, int sms);
cudaError_t launch_glr_fwd(const GlrParams &p, unsigned char *ws, int sms, cudaStream_t stream);
cudaError_t launch_glr_bwd(const GlrParams &p, unsigned char *ws, int sms, cudaStream_t stream);

// ------------------------------------------------------- layer norm
struct NormParams {
    const void *x;
    int64_t xs;
    const float *weight, *bias;    // null = 1, 0
    float eps;
    void *out;
    int64_t os;
    float *mean, *rstd;            // forward: null = not written
    int dtype;
    int64_t rows, D;
    // backward only
    const void *dout;
    int64_t ds;
    void *dx;                      // contiguous
    float *dweight, *dbias;        // null = not wanted
};
size_t norm_bwd_scratch_bytes(const NormParams &p, int sms);
cudaError_t launch_norm_fwd(const NormParams &p, int sms, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormParams &p, unsigned char *ws, int sms, cudaStream_t stream);

// ------------------------------------------------------- short causal convolution
struct ConvParams {
    const void *x;
    int64_t xs;
    const float *weight, *bias;    // weight [D, W]; bias may be null
    int W, silu;
    void *out;
    int64_t os;
    int dtype;
    const void *init;              // [N, W-1, D], dtype; null = zero rows
    void *fin;                     // [N, W-1, D], dtype; null = not written
    const int64_t *cu_seqlens;
    int64_t N, B, T, D, rows;
    // backward only
    const void *dout;
    int64_t ds;
    const float *dfinal;           // [N, W-1, D]
    void *dx;                      // contiguous
    float *dweight, *dbias, *dinit;   // dbias, dinit may be null
};
size_t conv_bwd_scratch_bytes(const ConvParams &p, int sms);
cudaError_t launch_conv_fwd(const ConvParams &p, int sms, cudaStream_t stream);
cudaError_t launch_conv_bwd(const ConvParams &p, unsigned char *ws, int sms, cudaStream_t stream);

// ------------------------------------------------------- RMS norm
struct RmsParams {
    const void *x, *res;           // res: null = no residual
    int64_t xs, rs;
    const float *weight;           // null = 1
    float eps;
    void *out;
    int64_t os;
    int out_dtype;                 // dtype, kE4M3 or kE5M2
    uint8_t *scales;               // 8-bit outputs: [rows, ceil(D/128)]
    int64_t ss;
    void *res_out;                 // null = the sum is not written
    int64_t ros;
    float *rstd;                   // forward: null = not written
    int dtype;
    int64_t rows, D;
    // backward only (x is the normed sum)
    const void *dout, *dres;       // dres: null = none
    int64_t ds, drs;
    void *dx;                      // contiguous
    float *dweight;                // null = not wanted
};
size_t rms_bwd_scratch_bytes(const RmsParams &p, int sms);
cudaError_t launch_rms_fwd(const RmsParams &p, int sms, cudaStream_t stream);
cudaError_t launch_rms_bwd(const RmsParams &p, unsigned char *ws, int sms, cudaStream_t stream);

// ------------------------------------------------------- 8-bit tensors
constexpr int kFp8Block = 128;     // elements of a row (and with `tile` rows) per scale

struct QuantParams {
    const void *x;                 // quantize: source; dequantize: destination
    int64_t xs;
    int dtype;
    void *q, *qt;                  // [rows, cols], [cols, rows]; either may be null
    int64_t qs, qts;
    uint8_t *s, *st;               // exponents + 127
    int64_t ss, sts;
    int q_dtype, tile;
    int64_t rows, cols;
};
cudaError_t launch_quantize(const QuantParams &p, int sms, cudaStream_t stream);
cudaError_t launch_dequantize(const QuantParams &p, int sms, cudaStream_t stream);

// out[m, n] = add[m, n] + sum_k a[m, k] b[n, k]
struct Fp8Operand {
    const void *q;                 // [rows, K], 16-byte aligned rows
    int64_t stride, rows;
    const uint8_t *s;              // [rows or ceil(rows/128), ceil(K/128)], 4-byte aligned rows
    int64_t s_stride;
    int tile, dtype;
};
struct MatmulParams {
    Fp8Operand a, b;
    void *out;
    int64_t os;
    const void *add;               // null = 0
    int64_t as;
    int dtype;
    int64_t K;
    int *err;
};
cudaError_t launch_matmul(const MatmulParams &p, int sms, cudaStream_t stream);

}  // namespace kda
