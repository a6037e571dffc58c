// Internal launch interface of the operators around the sequence layer, between the host layer
// (ttt_block_api.cu) and the kernels.
#pragma once

#include "ttt_internal.h"

namespace ttt {

// Root-mean-square norm over the residual stream (ttt_norm.cu).  `scale` set: 8-bit output.
constexpr int kNormMaxWidth = 16384;
struct NormArgs {
    int B, T, d;
    ttt_dtype dtype;
    float eps;
    const void *x, *residual;
    const float* weight;
    void *y, *h;
    float* scale;
};
struct NormBwdArgs {
    int B, T, d;
    ttt_dtype dtype;
    float eps;
    const void* h;
    const float* weight;
    const void *dy, *dh_in;
    void* dh;
    float* dweight;
};
cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t stream);
size_t rmsnorm_backward_workspace_bytes(int B, int T, int d, ttt_dtype dtype);
cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, float* workspace, cudaStream_t stream);
// out[c] = sum of partial[rows][cols] over the rows, in an order that the shape fixes
cudaError_t launch_column_sum(int rows, int cols, const float* partial, float* out, cudaStream_t stream);

// Short causal depthwise convolution (ttt_conv.cu)
constexpr int kConvMaxWidth = 4;
struct ConvArgs {
    int B, T, C, W;
    ttt_dtype dtype;
    int silu;
    long long ld;  // elements from one row of x to the next
    const void* x;
    const float *weight, *bias;
    const void* state0;
    const int* lengths;
    void *y, *state_T;
};
struct ConvBwdArgs {
    ConvArgs f;  // y, state_T unused
    const void *dy, *dstate_T;
    void* dx;
    float *dweight, *dbias;
    void* dstate0;
};
cudaError_t launch_conv(const ConvArgs& a, cudaStream_t stream);
size_t conv_backward_workspace_bytes(int B, int T, int C, int W);
cudaError_t launch_conv_backward(const ConvBwdArgs& a, float* workspace, cudaStream_t stream);

// Selective state space scan (ttt_ssm.cu, ttt_ssm_scan.cu, ttt_ssm_segments.cu, ttt_ssm_backward.cu)
constexpr int kSsmMaxStates = 64;
struct SsmArgs {
    int B, T, C, N;
    ttt_dtype dtype;
    int softplus;
    long long ld_u, ld_dt, ld_b, ld_c, ld_z;
    const void *u, *dt;
    const float *dt_bias, *A;
    const void *Bm, *Cm;
    const float* D;
    const void* z;
    const float* h0;
    const int* lengths;
    void* y;
    float* h_T;
};
struct SsmBwdArgs {
    SsmArgs f;  // y, h_T unused
    const void* dy;
    const float* dh_T;
    void *du, *ddt, *dz;
    float *dA, *dB, *dC, *dD, *ddt_bias, *dh0;
};
cudaError_t launch_ssm_forward(const SsmArgs& a, cudaStream_t stream);
// in place on h_T (= h0), any number of tokens
cudaError_t launch_ssm_token(const SsmArgs& a, cudaStream_t stream);
size_t ssm_backward_workspace_bytes(int B, int T, int C, int N);
cudaError_t launch_ssm_backward(const SsmBwdArgs& a, float* workspace, cudaStream_t stream);

// The 8-bit prologue (ttt_prologue_q8.cu): PrologueArgs with x and the weights in e4m3, the weights
// [H][d][d_model], and a scale a token and one an output feature.
struct PrologueScales {
    const float *x, *q, *k, *v, *lr;
};
bool prologue_q8_supports(int B, int T, int H, int d, int d_model);
cudaError_t launch_prologue_q8(const PrologueArgs& a, const PrologueScales& s, cudaStream_t stream);
cudaError_t read_and_clear_prologue_q8_error(unsigned int* out);

}  // namespace ttt
