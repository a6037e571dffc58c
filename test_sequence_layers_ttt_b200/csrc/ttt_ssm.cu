// Selective state space scan: the kernel for single tokens and a few, and the choice among the kernels for prompts.
//
//   dt = softplus(dt_raw + dt_bias) (or dt_raw + dt_bias),  h_t = e^(dt_t A) h_{t-1} + dt_t u_t B_t,
//   y_t = (sum_n C_t[n] h_t[n] + D u_t) silu(z_t)
// per channel, with N states a channel; B_t and C_t are shared by all channels of a token.
//
// For a token the state is nearly all there is to move (8 N bytes a channel, read and written), and for a
// few streams the launch is all there is to wait for.  Measured: one token of 64 streams of 2048 channels, 16 states
// (17 MB of state), 10 to 12 us replayed from a graph, 24 us a call with the host's share.
#include "ssm_params.cuh"

namespace ttt {
namespace {

using namespace ssm;

// Four neighbouring values of which the first `n` exist; kVec: all four, on a boundary of four
template <bool kVec, typename T>
__device__ __forceinline__ void load_four(const T* p, int n, float (&v)[kStates]) {
    if constexpr (kVec) {
        if (n > 0)
            load_vec<kStates>(p, v);
        else
            v[0] = v[1] = v[2] = v[3] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < kStates; i++) v[i] = i < n ? to_f32(p[i]) : 0.f;
    }
}

// A thread holds four states of one channel for the whole call; kLanes neighbouring lanes hold a
// channel, and y is their sum.  kVec: N is a multiple of four, and rows of B and C start on one.
template <typename T, int kLanes, bool kVec>
__global__ void __launch_bounds__(128) ttt_ssm_token_kernel(const Params p) {
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    const int part = threadIdx.x % kLanes;
    const long long bc = id / kLanes;
    const bool on = bc < (long long)p.B * p.C;
    const int b = on ? (int)(bc / p.C) : 0, c = on ? (int)(bc % p.C) : 0;
    const int n0 = part * kStates, live = on ? max(0, min(kStates, p.N - n0)) : 0;  // states that exist
    float h[kStates], a2[kStates];
    const size_t at = (size_t)bc * p.N + n0;
    if (p.h0)
        load_four<kVec>(p.h0 + at, live, h);
    else
        h[0] = h[1] = h[2] = h[3] = 0.f;
    const int len = length_of(p.lengths, b, p.T);
    load_four<kVec>(p.A + (size_t)c * p.N + n0, live, a2);
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f, skip = on && p.D ? p.D[c] : 0.f;
#pragma unroll
    for (int i = 0; i < kStates; i++) a2[i] = rate(a2[i]);
    for (int t = 0; t < p.T; t++) {
        const long long row = (long long)b * p.T + t;
        float Bt[kStates], Ct[kStates], dt = 0.f, u = 0.f, z = 0.f;
        const bool token = t < len;  // padding is not read, and a step of zero leaves the state
        load_four<kVec>(static_cast<const T*>(p.Bm) + row * p.ld_b + n0, token ? live : 0, Bt);
        load_four<kVec>(static_cast<const T*>(p.Cm) + row * p.ld_c + n0, token ? live : 0, Ct);
        if (on && token) {
            dt = to_f32(static_cast<const T*>(p.dt)[row * p.ld_dt + c]) + bias;
            u = to_f32(static_cast<const T*>(p.u)[row * p.ld_u + c]);
            if (p.z) z = to_f32(static_cast<const T*>(p.z)[row * p.ld_z + c]);
        }
        if (p.softplus) dt = ssm::softplus(dt);
        if (!token) dt = 0.f;
        const float du = dt * u;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < kStates; i++) {
            h[i] = fmaf(decay(dt * a2[i]), h[i], du * Bt[i]);
            y = fmaf(Ct[i], h[i], y);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (on && part == 0) {
            y = fmaf(skip, u, y);
            const float out[1] = {!token ? 0.f : p.z ? y * (z * sigmoid(z)) : y};
            store_vec<1>(static_cast<T*>(p.y) + row * p.C + c, out);
        }
    }
    if constexpr (kVec) {
        if (live > 0) store_vec<kStates>(p.h_T + at, h);
    } else {
#pragma unroll
        for (int i = 0; i < kStates; i++)
            if (i < live) p.h_T[at + i] = h[i];
    }
}

template <typename T>
cudaError_t launch_token(const SsmArgs& a, cudaStream_t stream) {
    const Params p = params_of(a);
    int lanes = 1;
    while (lanes * kStates < a.N) lanes *= 2;
    const long long blocks = ((long long)a.B * a.C * lanes + 127) / 128;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    const unsigned g = (unsigned)blocks;
    const auto four = [](const void* q, long long ld) {
        return reinterpret_cast<uintptr_t>(q) % (4 * sizeof(T)) == 0 && ld % 4 == 0;
    };
    if (a.N % 4 == 0 && four(a.Bm, a.ld_b) && four(a.Cm, a.ld_c)) {
        switch (lanes) {
            case 1: ttt_ssm_token_kernel<T, 1, true><<<g, 128, 0, stream>>>(p); break;
            case 2: ttt_ssm_token_kernel<T, 2, true><<<g, 128, 0, stream>>>(p); break;
            case 4: ttt_ssm_token_kernel<T, 4, true><<<g, 128, 0, stream>>>(p); break;
            case 8: ttt_ssm_token_kernel<T, 8, true><<<g, 128, 0, stream>>>(p); break;
            default: ttt_ssm_token_kernel<T, 16, true><<<g, 128, 0, stream>>>(p); break;
        }
        return cudaPeekAtLastError();
    }
    switch (lanes) {
        case 1: ttt_ssm_token_kernel<T, 1, false><<<g, 128, 0, stream>>>(p); break;
        case 2: ttt_ssm_token_kernel<T, 2, false><<<g, 128, 0, stream>>>(p); break;
        case 4: ttt_ssm_token_kernel<T, 4, false><<<g, 128, 0, stream>>>(p); break;
        case 8: ttt_ssm_token_kernel<T, 8, false><<<g, 128, 0, stream>>>(p); break;
        default: ttt_ssm_token_kernel<T, 16, false><<<g, 128, 0, stream>>>(p); break;
    }
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_ssm_token(const SsmArgs& a, cudaStream_t stream) {
    return a.dtype == TTT_BF16 ? launch_token<__nv_bfloat16>(a, stream) : launch_token<float>(a, stream);
}

cudaError_t launch_ssm_forward(const SsmArgs& a, cudaStream_t stream) {
    // A few tokens take the tokens' kernel: up to 8, or 24 where the others would have more than 37 blocks, whose start and
    // end cost as much as 24 tokens (14 x 7616 channels of 2 tokens 10 us against 74, of 24 tokens 50 against 76).
    // Blocks of 32 channels, one an SM.  Up to 37 of them (a quarter of 148 SMs) eight channels a block
    // still have an SM each, and those tiles, whose tokens are worked on side by side, take 61 clocks a
    // token against 87 (N = 16, bf16; 37 blocks of 4096 tokens: 132 us against 178).  Above 16 states the warps of a block
    // would hold too few registers for the other kernel.
    const long long blocks = (long long)a.B * ((a.C + 31) / 32);
    if (a.T <= (blocks <= 37 ? 8 : 24)) return launch_ssm_token(a, stream);
    if (blocks <= 37) return launch_ssm_segments(a, 8, stream);
    return a.N <= 16 ? launch_ssm_scan(a, stream) : launch_ssm_segments(a, 32, stream);
}

}  // namespace ttt
