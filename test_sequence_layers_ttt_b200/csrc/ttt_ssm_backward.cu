// Gradient of the selective state space scan.
//
// With dy' = dy silu(z) the gradient that reaches the scan's own output, and a_t = e^(dt_t A):
//   g_t = C_t dy'_t + a_{t+1} g_{t+1}          (g_T + the final state's gradient)
//   dC_t = sum over channels of dy'_t h_t,  dB_t = sum over channels of g_t dt_t u_t
//   du_t = dt_t (g_t . B_t) + D dy'_t,  ddt_t = (u_t (g_t . B_t) + sum_n g_t a_t h_{t-1} A) dt'(raw)
//   dA = sum_t g_t a_t h_{t-1} dt_t,  dD = sum_t dy'_t u_t,  dz_t = dy_t silu'(z_t) (C_t . h_t + D u_t)
//
// Two passes.  The first runs the scan and writes the state at the start of every chunk of kK tokens;
// the second takes the chunks from the last to the first: it recomputes a chunk's decays and states into
// registers and then walks it backwards.  A warp's lanes are 32 channels and a thread holds four states
// of one, so that B and C are one broadcast read each; the warps of a block share out the states.  Sums
// over states meet in shared memory, sums over the block's channels in shuffles; what is summed over
// blocks or sequences goes through the workspace and is added up in an order that the shape fixes.
#include "block_internal.h"
#include "ssm_math.cuh"
#include "vec_io.cuh"

namespace ttt {
namespace {

using namespace ssm;

constexpr int kS = 4;  // states a thread

struct SsmBwdParams {
    int B, T, C, N, chunks, cblocks;
    long long ld_u, ld_dt, ld_b, ld_c, ld_z;
    int softplus;
    const void *u, *dt, *Bm, *Cm, *z, *dy;
    const float *dt_bias, *A, *D, *h0, *dh_T;
    const int* lengths;
    void *du, *ddt, *dz;
    float* dh0;
    float* ckpt;     // [B][chunks][4 kNW][C]
    float* part_bc;  // [cblocks][B][T][2][N]
    float* part_c;   // [B][N + 2][C]: dA, dD, ddt_bias
};

// The block's 32 channels and sequence
struct Where {
    int b, c0;
};
__device__ __forceinline__ Where where(int cblocks) {
    return {(int)(blockIdx.x / cblocks), (int)(blockIdx.x % cblocks) * 32};
}

// ---------------------------------------------------------------- pass 1: the states at the chunks' starts
template <typename T, int kNW, int kK>
__global__ void __launch_bounds__(32 * kNW) ttt_ssm_checkpoint_kernel(const SsmBwdParams p) {
    constexpr int kNp = kS * kNW;                        // states, padded
    constexpr int kPairs = kK / kNW > 0 ? kK / kNW : 1;  // (token, channel) pairs a thread prepares
    __shared__ float2 s_dt[2][kK][32];                   // dt, dt u
    __shared__ __align__(16) float s_b[2][kK][kNp];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Where w = where(p.cblocks);
    const int c = w.c0 + lane;
    const bool on = c < p.C;
    const int len = length_of(p.lengths, w.b, p.T);
    const int n_chunks = (len + kK - 1) / kK;
    const int n0 = warp * kS;
    float h[kS], a2[kS];
#pragma unroll
    for (int i = 0; i < kS; i++) {
        const bool live = on && n0 + i < p.N;
        a2[i] = live ? p.A[(size_t)c * p.N + n0 + i] * kLog2e : 0.f;
        h[i] = live && p.h0 ? p.h0[((size_t)w.b * p.C + c) * p.N + n0 + i] : 0.f;
    }
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f;

    const auto fill = [&](int chunk, int buf) {
#pragma unroll
        for (int j = 0; j < kPairs; j++) {
            const int k = warp + j * kNW, t = chunk * kK + k;
            if (k < kK) {
                float dt = 0.f, du = 0.f;
                if (on && t < len) {
                    const long long row = (long long)w.b * p.T + t;
                    dt = to_f32(static_cast<const T*>(p.dt)[row * p.ld_dt + c]) + bias;
                    if (p.softplus) dt = ssm::softplus(dt);
                    du = dt * to_f32(static_cast<const T*>(p.u)[row * p.ld_u + c]);
                }
                s_dt[buf][k][lane] = make_float2(dt, du);
            }
        }
        for (int i = threadIdx.x; i < kK * kNp; i += 32 * kNW) {
            const int k = i / kNp, n = i % kNp, t = chunk * kK + k;
            float v = 0.f;
            if (t < len && n < p.N) v = to_f32(static_cast<const T*>(p.Bm)[((long long)w.b * p.T + t) * p.ld_b + n]);
            s_b[buf][k][n] = v;
        }
    };

    if (n_chunks > 0) fill(0, 0);
    __syncthreads();
    for (int chunk = 0; chunk < n_chunks; chunk++) {
        const int buf = chunk & 1;
        if (on) {
            float* out = p.ckpt + (((size_t)w.b * p.chunks + chunk) * kNp + n0) * p.C + c;
#pragma unroll
            for (int i = 0; i < kS; i++) out[(size_t)i * p.C] = h[i];
        }
        if (chunk + 1 < n_chunks) {
            fill(chunk + 1, buf ^ 1);
#pragma unroll
            for (int k = 0; k < kK; k++) {
                const float2 d = s_dt[buf][k][lane];
                const float4 Bt = *reinterpret_cast<const float4*>(&s_b[buf][k][n0]);
                const float bt[kS] = {Bt.x, Bt.y, Bt.z, Bt.w};
#pragma unroll
                for (int i = 0; i < kS; i++) h[i] = fmaf(decay(d.x * a2[i]), h[i], d.y * bt[i]);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- pass 2: the chunks, last to first

// 32 values a lane summed over the lanes: lane l returns the sum of value l.
__device__ __forceinline__ float sum_scatter(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; i++) {
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

template <int kNW, int kK>
struct BwdSmem {
    float b[kK][kS * kNW], c[kK][kS * kNW];
    float2 dt[kK][32];  // dt, dt u
    float dy[kK][32];   // dy'
    float gb[kNW][kK][32], ga[kNW][kK][32], y[kNW][kK][32];
    float sum[kNW][2][32];
};

template <typename T, int kNW, int kK>
__global__ void __launch_bounds__(32 * kNW) ttt_ssm_backward_kernel(const SsmBwdParams p) {
    constexpr int kNp = kS * kNW;
    constexpr int kPairs = kK / kNW > 0 ? kK / kNW : 1;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<kNW, kK>& s = *reinterpret_cast<BwdSmem<kNW, kK>*>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Where w = where(p.cblocks);
    const int cblk = (int)(blockIdx.x % p.cblocks);
    const int c = w.c0 + lane;
    const bool on = c < p.C;
    const int len = length_of(p.lengths, w.b, p.T);
    const int n_chunks = (len + kK - 1) / kK;
    const int n0 = warp * kS;
    float a2[kS], g[kS], dA[kS];
#pragma unroll
    for (int i = 0; i < kS; i++) {
        const bool live = on && n0 + i < p.N;
        a2[i] = live ? p.A[(size_t)c * p.N + n0 + i] * kLog2e : 0.f;
        g[i] = live && p.dh_T ? p.dh_T[((size_t)w.b * p.C + c) * p.N + n0 + i] : 0.f;
        dA[i] = 0.f;
    }
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f, skip = on && p.D ? p.D[c] : 0.f;
    float dD = 0.f, dbias = 0.f;

    // rows of padding: zero gradients
    for (int t = len + warp; t < p.T; t += kNW) {
        if (on) {
            const size_t at = ((size_t)w.b * p.T + t) * p.C + c;
            const float zero[1] = {0.f};
            store_vec<1>(static_cast<T*>(p.du) + at, zero);
            store_vec<1>(static_cast<T*>(p.ddt) + at, zero);
            if (p.dz) store_vec<1>(static_cast<T*>(p.dz) + at, zero);
        }
    }

    for (int chunk = n_chunks - 1; chunk >= 0; chunk--) {
        float u[kPairs], dt[kPairs], slope[kPairs], dyg[kPairs], dyz[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; j++) {
            const int k = warp + j * kNW, t = chunk * kK + k;
            u[j] = dt[j] = slope[j] = dyg[j] = dyz[j] = 0.f;
            if (k < kK) {
                if (on && t < len) {
                    const long long row = (long long)w.b * p.T + t;
                    const float raw = to_f32(static_cast<const T*>(p.dt)[row * p.ld_dt + c]) + bias;
                    u[j] = to_f32(static_cast<const T*>(p.u)[row * p.ld_u + c]);
                    dt[j] = p.softplus ? ssm::softplus(raw) : raw;
                    slope[j] = p.softplus ? sigmoid(raw) : 1.f;
                    dyg[j] = to_f32(static_cast<const T*>(p.dy)[row * p.C + c]);
                    if (p.z) {
                        const float z = to_f32(static_cast<const T*>(p.z)[row * p.ld_z + c]), sg = sigmoid(z);
                        dyz[j] = dyg[j] * sg * (1.f + z * (1.f - sg));
                        dyg[j] *= z * sg;
                    }
                }
                s.dt[k][lane] = make_float2(dt[j], dt[j] * u[j]);
                s.dy[k][lane] = dyg[j];
            }
        }
        for (int i = threadIdx.x; i < kK * kNp; i += 32 * kNW) {
            const int k = i / kNp, n = i % kNp, t = chunk * kK + k;
            const bool live = t < len && n < p.N;
            const long long row = (long long)w.b * p.T + t;
            s.b[k][n] = live ? to_f32(static_cast<const T*>(p.Bm)[row * p.ld_b + n]) : 0.f;
            s.c[k][n] = live ? to_f32(static_cast<const T*>(p.Cm)[row * p.ld_c + n]) : 0.f;
        }
        float a[kK][kS], h[kK + 1][kS];
        {
            const float* in = p.ckpt + (((size_t)w.b * p.chunks + chunk) * kNp + n0) * p.C + c;
#pragma unroll
            for (int i = 0; i < kS; i++) h[0][i] = on ? in[(size_t)i * p.C] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kK; k++) {
            const float2 d = s.dt[k][lane];
            const float4 Bt = *reinterpret_cast<const float4*>(&s.b[k][n0]);
            const float bt[kS] = {Bt.x, Bt.y, Bt.z, Bt.w};
#pragma unroll
            for (int i = 0; i < kS; i++) {
                a[k][i] = decay(d.x * a2[i]);
                h[k + 1][i] = fmaf(a[k][i], h[k][i], d.y * bt[i]);
            }
        }
#pragma unroll
        for (int k4 = kK - 4; k4 >= 0; k4 -= 4) {
            float v[32];  // of four tokens: dB and dC of the thread's four states
#pragma unroll
            for (int q = 3; q >= 0; q--) {
                const int k = k4 + q;
                const float2 d = s.dt[k][lane];
                const float dyk = s.dy[k][lane];
                const float4 Bt = *reinterpret_cast<const float4*>(&s.b[k][n0]);
                const float4 Ct = *reinterpret_cast<const float4*>(&s.c[k][n0]);
                const float bt[kS] = {Bt.x, Bt.y, Bt.z, Bt.w}, ct[kS] = {Ct.x, Ct.y, Ct.z, Ct.w};
                float gb = 0.f, ga = 0.f, y = 0.f;
#pragma unroll
                for (int i = 0; i < kS; i++) {
                    g[i] = fmaf(ct[i], dyk, g[i]);
                    v[q * 8 + i] = g[i] * d.y;
                    v[q * 8 + 4 + i] = dyk * h[k + 1][i];
                    gb = fmaf(g[i], bt[i], gb);
                    y = fmaf(ct[i], h[k + 1][i], y);
                    g[i] *= a[k][i];
                    const float x = g[i] * h[k][i];
                    ga = fmaf(x, a2[i], ga);
                    dA[i] = fmaf(x, d.x, dA[i]);
                }
                s.gb[warp][k][lane] = gb;
                s.ga[warp][k][lane] = ga;
                s.y[warp][k][lane] = y;
            }
            const float sum = sum_scatter(v, lane);
            const int t = chunk * kK + k4 + (lane >> 3), n = n0 + (lane & 3);
            if (t < len && n < p.N)
                p.part_bc[((((size_t)cblk * p.B + w.b) * p.T + t) * 2 + ((lane >> 2) & 1)) * p.N + n] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPairs; j++) {
            const int k = warp + j * kNW, t = chunk * kK + k;
            if (k < kK && on && t < len) {
                float gb = 0.f, ga = 0.f, y = 0.f;
#pragma unroll
                for (int q = 0; q < kNW; q++) {
                    gb += s.gb[q][k][lane];
                    ga += s.ga[q][k][lane];
                    y += s.y[q][k][lane];
                }
                const size_t at = ((size_t)w.b * p.T + t) * p.C + c;
                const float o_u[1] = {fmaf(dt[j], gb, skip * dyg[j])};
                const float o_dt[1] = {fmaf(u[j], gb, ga * (1.f / kLog2e)) * slope[j]};
                store_vec<1>(static_cast<T*>(p.du) + at, o_u);
                store_vec<1>(static_cast<T*>(p.ddt) + at, o_dt);
                if (p.dz) {
                    const float o_z[1] = {dyz[j] * fmaf(skip, u[j], y)};
                    store_vec<1>(static_cast<T*>(p.dz) + at, o_z);
                }
                dD = fmaf(dyg[j], u[j], dD);
                dbias += o_dt[0];
            }
        }
    }
    s.sum[warp][0][lane] = dD;
    s.sum[warp][1][lane] = dbias;
    __syncthreads();
    if (on) {
#pragma unroll
        for (int i = 0; i < kS; i++) {
            if (n0 + i < p.N) {
                p.part_c[((size_t)w.b * (p.N + 2) + n0 + i) * p.C + c] = dA[i];
                if (p.dh0) p.dh0[((size_t)w.b * p.C + c) * p.N + n0 + i] = g[i];
            }
        }
        if (warp == 0) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int q = 0; q < kNW; q++) {
                x += s.sum[q][0][lane];
                y += s.sum[q][1][lane];
            }
            p.part_c[((size_t)w.b * (p.N + 2) + p.N) * p.C + c] = x;
            p.part_c[((size_t)w.b * (p.N + 2) + p.N + 1) * p.C + c] = y;
        }
    }
}

// ---------------------------------------------------------------- the sums over blocks and sequences
__global__ void __launch_bounds__(256) ttt_ssm_bc_sum_kernel(int B, int T, int N, int cblocks, const int* lengths,
                                                             const float* __restrict__ part, float* __restrict__ dB,
                                                             float* __restrict__ dC) {
    const size_t per = (size_t)T * 2 * N, total = (size_t)B * per;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int b = (int)(i / per);
    const size_t r = i % per;
    const int t = (int)(r / (2 * N)), m = (int)(r % (2 * N));
    float a = 0.f;
    if (t < length_of(lengths, b, T))
        for (int k = 0; k < cblocks; k++) a += part[(size_t)k * total + i];
    (m < N ? dB : dC)[((size_t)b * T + t) * N + (m < N ? m : m - N)] = a;
}

__global__ void __launch_bounds__(256) ttt_ssm_channel_sum_kernel(int B, int C, int N, const float* __restrict__ part,
                                                                  float* __restrict__ dA, float* __restrict__ dD,
                                                                  float* __restrict__ dbias) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (size_t)(N + 2) * C) return;
    const int n = (int)(i / C), c = (int)(i % C);
    float a = 0.f;
    for (int b = 0; b < B; b++) a += part[(size_t)b * (N + 2) * C + i];
    if (n < N)
        dA[(size_t)c * N + n] = a;
    else if (n == N) {
        if (dD) dD[c] = a;
    } else if (dbias) {
        dbias[c] = a;
    }
}

constexpr int warps_for(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
// 16 tokens a chunk keep 128 values in registers; with 16 warps a thread has 128 registers, so 8 there
constexpr int chunk_for(int kNW) { return kNW <= 8 ? 16 : 8; }

struct Layout {
    size_t ckpt, part_bc, part_c, total;  // floats
};
Layout layout(int B, int T, int C, int N) {
    const int nw = warps_for(N), K = chunk_for(nw);
    const size_t chunks = ((size_t)T + K - 1) / K, cblocks = ((size_t)C + 31) / 32;
    const auto up = [](size_t x) { return (x + 3) / 4 * 4; };
    Layout l{};
    l.ckpt = up((size_t)B * chunks * kS * nw * C);
    l.part_bc = up(cblocks * B * T * 2 * N);
    l.part_c = up((size_t)B * (N + 2) * C);
    l.total = l.ckpt + l.part_bc + l.part_c;
    return l;
}

template <typename T, int kNW>
cudaError_t launch(const SsmBwdParams& p, cudaStream_t stream) {
    constexpr int kK = chunk_for(kNW);
    const unsigned grid = (unsigned)((long long)p.B * p.cblocks);
    ttt_ssm_checkpoint_kernel<T, kNW, kK><<<grid, 32 * kNW, 0, stream>>>(p);
    cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess) return e;
    constexpr int smem = (int)sizeof(BwdSmem<kNW, kK>);
    e = cudaFuncSetAttribute(ttt_ssm_backward_kernel<T, kNW, kK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ttt_ssm_backward_kernel<T, kNW, kK><<<grid, 32 * kNW, smem, stream>>>(p);
    return cudaPeekAtLastError();
}

template <typename T>
cudaError_t dispatch(const SsmBwdParams& p, cudaStream_t stream) {
    switch (warps_for(p.N)) {
        case 1: return launch<T, 1>(p, stream);
        case 2: return launch<T, 2>(p, stream);
        case 4: return launch<T, 4>(p, stream);
        case 8: return launch<T, 8>(p, stream);
        default: return launch<T, 16>(p, stream);
    }
}

}  // namespace

size_t ssm_backward_workspace_bytes(int B, int T, int C, int N) {
    if (B < 1 || T < 0 || C < 1 || N < 1 || N > kSsmMaxStates) return 0;
    return layout(B, T, C, N).total * sizeof(float);
}

cudaError_t launch_ssm_backward(const SsmBwdArgs& a, float* workspace, cudaStream_t stream) {
    const SsmArgs& f = a.f;
    const Layout l = layout(f.B, f.T, f.C, f.N);
    SsmBwdParams p{};
    p.B = f.B;
    p.T = f.T;
    p.C = f.C;
    p.N = f.N;
    const int K = chunk_for(warps_for(f.N));
    p.chunks = (f.T + K - 1) / K;
    p.cblocks = (f.C + 31) / 32;
    if ((long long)p.B * p.cblocks >= (1LL << 31)) return cudaErrorInvalidValue;
    p.ld_u = f.ld_u;
    p.ld_dt = f.ld_dt;
    p.ld_b = f.ld_b;
    p.ld_c = f.ld_c;
    p.ld_z = f.ld_z;
    p.softplus = f.softplus;
    p.u = f.u;
    p.dt = f.dt;
    p.Bm = f.Bm;
    p.Cm = f.Cm;
    p.z = f.z;
    p.dy = a.dy;
    p.dt_bias = f.dt_bias;
    p.A = f.A;
    p.D = f.D;
    p.h0 = f.h0;
    p.dh_T = a.dh_T;
    p.lengths = f.lengths;
    p.du = a.du;
    p.ddt = a.ddt;
    p.dz = a.dz;
    p.dh0 = a.dh0;
    p.ckpt = workspace;
    p.part_bc = workspace + l.ckpt;
    p.part_c = p.part_bc + l.part_bc;
    cudaError_t e = f.dtype == TTT_BF16 ? dispatch<__nv_bfloat16>(p, stream) : dispatch<float>(p, stream);
    if (e != cudaSuccess) return e;
    const size_t bc = (size_t)f.B * f.T * 2 * f.N;
    if (bc > 0) {
        ttt_ssm_bc_sum_kernel<<<(unsigned)((bc + 255) / 256), 256, 0, stream>>>(f.B, f.T, f.N, p.cblocks, f.lengths,
                                                                                p.part_bc, a.dB, a.dC);
        e = cudaPeekAtLastError();
        if (e != cudaSuccess) return e;
    }
    const size_t ch = (size_t)(f.N + 2) * f.C;
    ttt_ssm_channel_sum_kernel<<<(unsigned)((ch + 255) / 256), 256, 0, stream>>>(f.B, f.C, f.N, p.part_c, a.dA, a.dD,
                                                                                 a.ddt_bias);
    return cudaPeekAtLastError();
}

}  // namespace ttt
