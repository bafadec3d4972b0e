// Launch parameters shared by the host entry points (layer_api.cu) and the kernels of the
// operators around the delta rule: the gated linear recurrence (glr*.cu), layer norm
// (layer_norm.cu) and the short causal convolution (short_conv.cu).  Not part of the
// public ABI (that is include/kda.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kda_internal.h"

namespace kda {

// Element types of the operators' tensors (KDA_DTYPE_* of include/kda.h).
enum DType : int { kBF16 = 1, kFP32 = 2, kFP16 = 3 };

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

}  // namespace kda
