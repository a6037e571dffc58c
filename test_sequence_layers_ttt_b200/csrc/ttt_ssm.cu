// Selective state space scan: the kernel for single tokens, and the choice among the kernels for prompts.
//
//   dt = softplus(dt_raw + dt_bias) (or dt_raw + dt_bias),  h_t = e^(dt_t A) h_{t-1} + dt_t u_t B_t,
//   y_t = (sum_n C_t[n] h_t[n] + D u_t) silu(z_t)
// per channel, with N states a channel; B_t and C_t are shared by all channels of a token.
//
// For a token the state is nearly all there is to move (8 N bytes a channel, read and written), and for a
// few streams the launch is all there is to wait for.
#include "ssm_params.cuh"

namespace ttt {
namespace {

using namespace ssm;

// A thread holds four states of one channel for the whole call; kLanes neighbouring lanes hold a
// channel, and y is their sum.
template <typename T, int kLanes>
__global__ void __launch_bounds__(128) ttt_ssm_token_kernel(const Params p) {
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    const int part = threadIdx.x % kLanes;
    const long long bc = id / kLanes;
    const bool on = bc < (long long)p.B * p.C;
    const int b = on ? (int)(bc / p.C) : 0, c = on ? (int)(bc % p.C) : 0;
    const int n0 = part * kStates;
    const int len = on ? length_of(p.lengths, b, p.T) : 0;
    float h[kStates], a2[kStates];
#pragma unroll
    for (int i = 0; i < kStates; i++) {
        const bool live = on && n0 + i < p.N;
        a2[i] = live ? p.A[(size_t)c * p.N + n0 + i] * kLog2e : 0.f;
        h[i] = live && p.h0 ? p.h0[(size_t)bc * p.N + n0 + i] : 0.f;
    }
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f, skip = on && p.D ? p.D[c] : 0.f;
    for (int t = 0; t < p.T; t++) {
        const long long row = (long long)b * p.T + t;
        float y = 0.f, u = 0.f;
        if (t < len) {
            float dt = to_f32(static_cast<const T*>(p.dt)[row * p.ld_dt + c]) + bias;
            if (p.softplus) dt = ssm::softplus(dt);
            u = to_f32(static_cast<const T*>(p.u)[row * p.ld_u + c]);
            const float du = dt * u;
            const T* Bt = static_cast<const T*>(p.Bm) + row * p.ld_b;
            const T* Ct = static_cast<const T*>(p.Cm) + row * p.ld_c;
#pragma unroll
            for (int i = 0; i < kStates; i++) {
                if (n0 + i < p.N) {
                    h[i] = fmaf(decay(dt * a2[i]), h[i], du * to_f32(Bt[n0 + i]));
                    y = fmaf(to_f32(Ct[n0 + i]), h[i], y);
                }
            }
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (on && part == 0) {
            if (t < len) {
                y = fmaf(skip, u, y);
                if (p.z) {
                    const float z = to_f32(static_cast<const T*>(p.z)[row * p.ld_z + c]);
                    y *= z * sigmoid(z);
                }
            }
            const float out[1] = {y};
            store_vec<1>(static_cast<T*>(p.y) + row * p.C + c, out);
        }
    }
#pragma unroll
    for (int i = 0; i < kStates; i++)
        if (on && n0 + i < p.N) p.h_T[(size_t)bc * p.N + n0 + i] = h[i];
}

template <typename T>
cudaError_t launch_token(const SsmArgs& a, cudaStream_t stream) {
    const Params p = params_of(a);
    int lanes = 1;
    while (lanes * kStates < a.N) lanes *= 2;
    const long long blocks = ((long long)a.B * a.C * lanes + 127) / 128;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    const unsigned g = (unsigned)blocks;
    switch (lanes) {
        case 1: ttt_ssm_token_kernel<T, 1><<<g, 128, 0, stream>>>(p); break;
        case 2: ttt_ssm_token_kernel<T, 2><<<g, 128, 0, stream>>>(p); break;
        case 4: ttt_ssm_token_kernel<T, 4><<<g, 128, 0, stream>>>(p); break;
        case 8: ttt_ssm_token_kernel<T, 8><<<g, 128, 0, stream>>>(p); break;
        default: ttt_ssm_token_kernel<T, 16><<<g, 128, 0, stream>>>(p); break;
    }
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_ssm_token(const SsmArgs& a, cudaStream_t stream) {
    return a.dtype == TTT_BF16 ? launch_token<__nv_bfloat16>(a, stream) : launch_token<float>(a, stream);
}

size_t ssm_forward_workspace_bytes(int, int, int, int) { return 0; }

cudaError_t launch_ssm_forward(const SsmArgs& a, float*, cudaStream_t stream) {
    // Blocks of 32 channels, one an SM.  Up to 37 of them (a quarter of 148 SMs) eight channels a block
    // still have an SM each, and those tiles, whose tokens are worked on side by side, take 61 clocks a
    // token against 87 (N = 16, bf16).  Above 16 states the warps of a block would hold too few registers
    // for the other kernel.
    const long long blocks = (long long)a.B * ((a.C + 31) / 32);
    if (blocks <= 37) return launch_ssm_segments(a, 8, stream);
    return a.N <= 16 ? launch_ssm_scan(a, stream) : launch_ssm_segments(a, 32, stream);
}

}  // namespace ttt
