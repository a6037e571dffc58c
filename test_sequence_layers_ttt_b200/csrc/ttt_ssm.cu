// Selective state space scan, forward and token by token.
//
//   dt = softplus(dt_raw + dt_bias) (or dt_raw + dt_bias),  h_t = e^(dt_t A) h_{t-1} + dt_t u_t B_t,
//   y_t = (sum_n C_t[n] h_t[n] + D u_t) silu(z_t)
// per channel, with kN states a channel; B_t and C_t are shared by all channels of a token.
#include "block_internal.h"
#include "ssm_math.cuh"
#include "vec_io.cuh"

namespace ttt {
namespace {

using namespace ssm;

struct SsmParams {
    int B, T, C, N;
    long long ld_u, ld_dt, ld_b, ld_c, ld_z;
    int softplus;
    const void *u, *dt, *Bm, *Cm, *z;
    const float *dt_bias, *A, *D;
    const float* h0;
    const int* lengths;
    void* y;
    float* h_T;
};

constexpr int kStates = 4;  // states a thread

// A thread holds four states of one channel for the whole call; kLanes neighbouring lanes hold a
// channel, and y is their sum.
template <typename T, int kLanes>
__global__ void __launch_bounds__(128) ttt_ssm_token_kernel(const SsmParams p) {
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

SsmParams params_of(const SsmArgs& a) {
    SsmParams p{};
    p.B = a.B;
    p.T = a.T;
    p.C = a.C;
    p.N = a.N;
    p.ld_u = a.ld_u;
    p.ld_dt = a.ld_dt;
    p.ld_b = a.ld_b;
    p.ld_c = a.ld_c;
    p.ld_z = a.ld_z;
    p.softplus = a.softplus;
    p.u = a.u;
    p.dt = a.dt;
    p.Bm = a.Bm;
    p.Cm = a.Cm;
    p.z = a.z;
    p.dt_bias = a.dt_bias;
    p.A = a.A;
    p.D = a.D;
    p.h0 = a.h0;
    p.lengths = a.lengths;
    p.y = a.y;
    p.h_T = a.h_T;
    return p;
}

// ---------------------------------------------------------------- prompts
constexpr int kSeg = 16;       // tokens a warp takes of a tile
constexpr int kMaxWarps = 8;   // warps a block
constexpr size_t kMaxSmem = 227 * 1024;

// Shared memory of the scan, for tiles of `tile` tokens: raw rows of the tile in work and of the next one,
// B and C as floats, A log2(e), the state that goes from tile to tile, the segments' ends and decays.
template <typename T, int kL>
struct ScanSmem {
    float4 *end, *fall;  // [2][kMaxWarps][32]
    float4 *a2, *h;      // [groups][32]; [2][groups][32]
    float *b, *c;        // [tile][n_pad]
    T *u, *dt, *z;       // [2][tile][kL]
    T *rb, *rc;          // [2][tile][n_pad]

    __host__ __device__ static size_t bytes(int tile, int n_pad) {
        const size_t groups = n_pad / (kStates * (32 / kL));
        return (4 * kMaxWarps + 3 * groups) * 32 * sizeof(float4) +
               (size_t)tile * (n_pad * (2 * sizeof(float) + 4 * sizeof(T)) + 6 * kL * sizeof(T));
    }
    __device__ ScanSmem(unsigned char* raw, int tile, int n_pad) {
        const int groups = n_pad / (kStates * (32 / kL));
        end = reinterpret_cast<float4*>(raw);
        fall = end + 2 * kMaxWarps * 32;
        a2 = fall + 2 * kMaxWarps * 32;
        h = a2 + groups * 32;
        b = reinterpret_cast<float*>(h + 2 * groups * 32);
        c = b + tile * n_pad;
        u = reinterpret_cast<T*>(c + tile * n_pad);
        dt = u + 2 * tile * kL;
        z = dt + 2 * tile * kL;
        rb = z + 2 * tile * kL;
        rc = rb + 2 * tile * n_pad;
    }
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool live) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// Rows [t0, t0 + rows) of `cols` columns into shared memory (row stride `cols`); rows at or past `len` and
// columns at or past `width` become zeros.
template <typename T, bool kVec>
__device__ __forceinline__ void stage_rows(T* dst, const T* src, long long ld, int t0, int rows, int len, int cols, int width,
                                           int tid, int threads) {
    constexpr int kV = kVec ? 16 / (int)sizeof(T) : 1;
    const int per = cols / kV;
    for (int i = tid; i < rows * per; i += threads) {
        const int r = i / per, c = (i % per) * kV;
        const bool live = t0 + r < len && c < width;
        if constexpr (kVec) {
            copy16(dst + r * cols + c, live ? src + (long long)(t0 + r) * ld + c : src, live);
        } else {
            dst[r * cols + c] = live ? src[(long long)(t0 + r) * ld + c] : T(0.f);
        }
    }
}

// A block takes kL channels of one sequence, tile by tile; a warp takes kSeg tokens of the tile for all of
// them, with kQ = 32 / kL lanes a channel sharing out the states in fours.  Per four states a thread
// computes its tokens' decays and inputs into registers and runs them from zero; the ends and the decays
// over the whole segments go through shared memory, every warp folds those before its own onto the tile's
// first state, and runs its tokens again from there.  So the special functions, the bound, are evaluated
// once a token and state, and a sequence keeps 32 warps' worth of work in flight for every 32 channels.
template <typename T, int kL, bool kVecRows, bool kVecBC>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) ttt_ssm_scan_kernel(const SsmParams p, const int cblocks, const int n_pad) {
    constexpr int kQ = 32 / kL;
    constexpr int kOwn = kSeg / kQ;  // tokens whose elementwise work a lane does
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    const int b = (int)(blockIdx.x / cblocks), c0 = (int)(blockIdx.x % cblocks) * kL;
    const int ch = lane / kQ, part = lane % kQ, c = c0 + ch;
    const bool on = c < p.C;
    const int len = length_of(p.lengths, b, p.T);
    const int tile = kSeg * warps, groups = n_pad / (kStates * kQ);
    const ScanSmem<T, kL> s(smem_raw, tile, n_pad);
    const T* u_rows = static_cast<const T*>(p.u) + (long long)b * p.T * p.ld_u + c0;
    const T* dt_rows = static_cast<const T*>(p.dt) + (long long)b * p.T * p.ld_dt + c0;
    const T* z_rows = static_cast<const T*>(p.z) + (long long)b * p.T * p.ld_z + c0;
    const T* b_rows = static_cast<const T*>(p.Bm) + (long long)b * p.T * p.ld_b;
    const T* c_rows = static_cast<const T*>(p.Cm) + (long long)b * p.T * p.ld_c;
    T* y_rows = static_cast<T*>(p.y) + (long long)b * p.T * p.C + c;

    const auto stage = [&](int t0, int buf) {
        const int width = p.C - c0;
        stage_rows<T, kVecRows>(s.u + buf * tile * kL, u_rows, p.ld_u, t0, tile, len, kL, width, tid, threads);
        stage_rows<T, kVecRows>(s.dt + buf * tile * kL, dt_rows, p.ld_dt, t0, tile, len, kL, width, tid, threads);
        if (p.z) stage_rows<T, kVecRows>(s.z + buf * tile * kL, z_rows, p.ld_z, t0, tile, len, kL, width, tid, threads);
        stage_rows<T, kVecBC>(s.rb + buf * tile * n_pad, b_rows, p.ld_b, t0, tile, len, n_pad, p.N, tid, threads);
        stage_rows<T, kVecBC>(s.rc + buf * tile * n_pad, c_rows, p.ld_c, t0, tile, len, n_pad, p.N, tid, threads);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    for (int g = warp; g < groups; g += warps) {
        float h[kStates], v[kStates];
#pragma unroll
        for (int i = 0; i < kStates; i++) {
            const int n = (g * kQ + part) * kStates + i;
            h[i] = on && n < p.N && p.h0 ? p.h0[((size_t)b * p.C + c) * p.N + n] : 0.f;
            v[i] = on && n < p.N ? p.A[(size_t)c * p.N + n] * kLog2e : 0.f;
        }
        s.h[g * 32 + lane] = make_float4(h[0], h[1], h[2], h[3]);
        s.a2[g * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
    }
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f, skip = on && p.D ? p.D[c] : 0.f;

    if (len > 0) stage(0, 0);
    int turn = 0, buf = 0;  // turn: which of the two segment buffers
    for (int t0 = 0; t0 < len; t0 += tile, buf ^= 1) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (t0 + tile < len) stage(t0 + tile, buf ^ 1);
        for (int i = tid; i < tile * n_pad; i += threads) {
            s.b[i] = to_f32(s.rb[buf * tile * n_pad + i]);
            s.c[i] = to_f32(s.rc[buf * tile * n_pad + i]);
        }
        const int k0 = warp * kSeg;
        float dt[kSeg], du[kSeg], y[kSeg], own_u[kOwn];
        {
            float own_dt[kOwn];
#pragma unroll
            for (int j = 0; j < kOwn; j++) {
                const int k = k0 + part * kOwn + j;
                float d = to_f32(s.dt[(buf * tile + k) * kL + ch]) + bias;
                if (p.softplus) d = ssm::softplus(d);
                own_dt[j] = t0 + k < len ? d : 0.f;
                own_u[j] = to_f32(s.u[(buf * tile + k) * kL + ch]);
            }
#pragma unroll
            for (int k = 0; k < kSeg; k++) {
                y[k] = 0.f;
                if constexpr (kQ == 1) {
                    dt[k] = own_dt[k];
                    du[k] = own_dt[k] * own_u[k];
                } else {
                    const int from = (lane & ~(kQ - 1)) + k / kOwn;
                    dt[k] = __shfl_sync(0xffffffffu, own_dt[k % kOwn], from);
                    du[k] = __shfl_sync(0xffffffffu, own_dt[k % kOwn] * own_u[k % kOwn], from);
                }
            }
        }
        float sum_dt = 0.f;
#pragma unroll
        for (int k = 0; k < kSeg; k++) sum_dt += dt[k];
        __syncthreads();
        for (int g = 0; g < groups; g++, turn ^= 1) {
            const int n0 = (g * kQ + part) * kStates;
            const ulonglong2 a2 = *reinterpret_cast<const ulonglong2*>(&s.a2[g * 32 + lane]);
            f2 a[kSeg][2], x[kSeg][2], h[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < kSeg; k++) {
                const ulonglong2 Bt = *reinterpret_cast<const ulonglong2*>(&s.b[(k0 + k) * n_pad + n0]);
                const f2 d2 = pack2(dt[k], dt[k]), u2 = pack2(du[k], du[k]);
                a[k][0] = decay2(mul2(d2, a2.x));
                a[k][1] = decay2(mul2(d2, a2.y));
                x[k][0] = mul2(u2, Bt.x);
                x[k][1] = mul2(u2, Bt.y);
                h[0] = fma2(a[k][0], h[0], x[k][0]);
                h[1] = fma2(a[k][1], h[1], x[k][1]);
            }
            const f2 s2 = pack2(sum_dt, sum_dt);
            const f2 f0 = decay2(mul2(s2, a2.x)), f1 = decay2(mul2(s2, a2.y));
            *reinterpret_cast<ulonglong2*>(&s.end[(turn * kMaxWarps + warp) * 32 + lane]) = make_ulonglong2(h[0], h[1]);
            *reinterpret_cast<ulonglong2*>(&s.fall[(turn * kMaxWarps + warp) * 32 + lane]) = make_ulonglong2(f0, f1);
            __syncthreads();
            const ulonglong2 first = reinterpret_cast<const ulonglong2*>(s.h)[(buf * groups + g) * 32 + lane];
            h[0] = first.x;
            h[1] = first.y;
            for (int v = 0; v < warp; v++) {
                const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(&s.end[(turn * kMaxWarps + v) * 32 + lane]);
                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&s.fall[(turn * kMaxWarps + v) * 32 + lane]);
                h[0] = fma2(f.x, h[0], e.x);
                h[1] = fma2(f.y, h[1], e.y);
            }
#pragma unroll
            for (int k = 0; k < kSeg; k++) {
                const ulonglong2 Ct = *reinterpret_cast<const ulonglong2*>(&s.c[(k0 + k) * n_pad + n0]);
                h[0] = fma2(a[k][0], h[0], x[k][0]);
                h[1] = fma2(a[k][1], h[1], x[k][1]);
                float lo, hi;
                unpack2(fma2(Ct.y, h[1], mul2(Ct.x, h[0])), lo, hi);
                y[k] += lo + hi;
            }
            if (warp == warps - 1)
                reinterpret_cast<ulonglong2*>(s.h)[((buf ^ 1) * groups + g) * 32 + lane] = make_ulonglong2(h[0], h[1]);
        }
        // a channel's lanes share out the tokens: kOwn sums each
        float own_y[kOwn];
        if constexpr (kQ == 1) {
#pragma unroll
            for (int j = 0; j < kOwn; j++) own_y[j] = y[j];
        } else {
            static_assert(kQ == 1 || kQ == 4, "two exchange steps");
            const bool up2 = part & 2, up1 = part & 1;
            float half[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float keep = up2 ? y[8 + j] : y[j], send = up2 ? y[j] : y[8 + j];
                half[j] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float keep = up1 ? half[4 + j] : half[j], send = up1 ? half[j] : half[4 + j];
                own_y[j] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
            }
        }
#pragma unroll
        for (int j = 0; j < kOwn; j++) {
            const int k = k0 + part * kOwn + j, t = t0 + k;
            float o[1] = {fmaf(skip, own_u[j], own_y[j])};
            if (p.z) {
                const float z = to_f32(s.z[(buf * tile + k) * kL + ch]);
                o[0] *= z * sigmoid(z);
            }
            if (on && t < len) store_vec<1>(y_rows + (long long)t * p.C, o);
        }
    }
    __syncthreads();
    for (int g = warp; g < groups; g += warps) {
        const float4 v = s.h[(buf * groups + g) * 32 + lane];
        const float h[kStates] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < kStates; i++) {
            const int n = (g * kQ + part) * kStates + i;
            if (on && n < p.N) p.h_T[((size_t)b * p.C + c) * p.N + n] = h[i];
        }
    }
    const float zero[1] = {0.f};
    for (int t = len + warp * kQ + part; t < p.T; t += warps * kQ)
        if (on) store_vec<1>(y_rows + (long long)t * p.C, zero);
}

bool rows16(const void* q, long long ld, int width, int es) {
    return !q || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (ld * es) % 16 == 0 && (width * es) % 16 == 0);
}

template <typename T, int kL>
cudaError_t launch_scan(const SsmArgs& a, cudaStream_t stream) {
    const SsmParams p = params_of(a);
    constexpr int es = sizeof(T), step = kStates * (32 / kL);
    const int n_pad = (a.N + step - 1) / step * step;
    const long long cblocks = (a.C + kL - 1) / kL, grid = a.B * cblocks;
    if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
    // a warp for every 16 tokens, up to 8, and fewer where many states make the tile too large
    const int segs = (a.T + kSeg - 1) / kSeg;
    int warps = segs < 1 ? 1 : (segs < kMaxWarps ? segs : kMaxWarps);
    while (warps > 1 && ScanSmem<T, kL>::bytes(kSeg * warps, n_pad) > kMaxSmem) warps--;
    const bool rows = rows16(a.u, a.ld_u, a.C, es) && rows16(a.dt, a.ld_dt, a.C, es) && rows16(a.z, a.ld_z, a.C, es);
    const bool bc = rows16(a.Bm, a.ld_b, a.N, es) && rows16(a.Cm, a.ld_c, a.N, es);
    const size_t smem = ScanSmem<T, kL>::bytes(kSeg * warps, n_pad);
    const auto run = [&](auto kernel) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)grid, 32 * warps, smem, stream>>>(p, (int)cblocks, n_pad);
        return cudaPeekAtLastError();
    };
    if (rows && bc) return run(ttt_ssm_scan_kernel<T, kL, true, true>);
    if (rows) return run(ttt_ssm_scan_kernel<T, kL, true, false>);
    return run(ttt_ssm_scan_kernel<T, kL, false, false>);
}

template <typename T>
cudaError_t launch_prompt(const SsmArgs& a, cudaStream_t stream) {
    // few channels: eight a block, so that four times as many SMs have one
    return (long long)a.B * ((a.C + 31) / 32) <= 74 ? launch_scan<T, 8>(a, stream) : launch_scan<T, 32>(a, stream);
}

template <typename T>
cudaError_t launch_token(const SsmArgs& a, cudaStream_t stream) {
    const SsmParams p = params_of(a);
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
    return a.dtype == TTT_BF16 ? launch_prompt<__nv_bfloat16>(a, stream) : launch_prompt<float>(a, stream);
}

}  // namespace ttt
