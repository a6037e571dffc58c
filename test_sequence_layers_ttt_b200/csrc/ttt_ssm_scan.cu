// Selective scan with the states shared out among the warps of a block, for launches with enough channels.
//
// A block takes 32 channels (a warp's lanes) of one sequence and walks its tokens; kWarps warps hold four
// states a thread, so that B and C are broadcast reads and nothing is computed twice.  kHelpers more warps do
// what is elementwise beside them: they bring the next tiles' rows in, evaluate the softplus, lay B and C out
// as floats with a state's tokens side by side (for the packed fp32 instructions, which take tokens in
// pairs), and finish the last tile: the sum over the warps, D, the gate, the store.  One barrier a tile.
//
// Per token and 32 channels of 16 states an SM has 20 special-function results a channel (40 clocks), and on
// each of its four schedulers 29 instructions of the recursion (34 clocks of the fp32 pipe); by the rate of issue the
// helpers have some 25.  Measured: 1.41 ms, 89 clocks a token (1.3B width, 32k tokens, bf16; fp32 95), in 63 % of
// which a scheduler issues; the recursion alone took 75, as it waits on its own results: two channels a thread would
// hide that but leave half of the SMs idle.
#include "ssm_params.cuh"

#include <type_traits>

namespace ttt {
namespace {

using namespace ssm;

constexpr int kHelpers = 8;

// Shared memory.  What the helpers prepare for the recursion and what the recursion leaves them is double-
// buffered; raw rows are in four buffers, of the tile being finished, in work, being prepared and on its way.
template <typename T>
struct ScanSmem {
    static constexpr int kTile = sizeof(T) == 2 ? 64 : 32;  // tokens of a tile; fp32 rows leave room for 32
    static constexpr int kQuads = kTile / 4;  // a thread's unit of work: four tokens of a channel
    static constexpr int kPitch = kTile + 4;  // of a state's row of B or C
    float4 *dt, *du;  // [2][kQuads][32]: steps and inputs of a channel's four tokens
    float4* y;        // [2][warps][kQuads][32]: each warp's part of the sum over the states
    float *b, *c;     // [2][n_pad][kPitch]: a state's tokens side by side
    T *u, *raw, *z;   // [4][kTile][32]; raw: dt as it was given
    T *rb, *rc;       // [4][kTile][n_pad]

    __host__ __device__ static constexpr size_t bytes(int warps, int n_pad) {
        return 2 * (2 + warps) * kQuads * 32 * sizeof(float4) + 4 * (size_t)n_pad * kPitch * sizeof(float) +
               4 * kTile * (size_t)(3 * 32 + 2 * n_pad) * sizeof(T);
    }
    __device__ ScanSmem(unsigned char* at, int warps, int n_pad) {
        dt = reinterpret_cast<float4*>(at);
        du = dt + 2 * kQuads * 32;
        y = du + 2 * kQuads * 32;
        b = reinterpret_cast<float*>(y + 2 * warps * kQuads * 32);
        c = b + 2 * n_pad * kPitch;
        u = reinterpret_cast<T*>(c + 2 * n_pad * kPitch);
        raw = u + 4 * kTile * 32;
        z = raw + 4 * kTile * 32;
        rb = z + 4 * kTile * 32;
        rc = rb + 4 * kTile * n_pad;
    }
};

template <typename T, int kWarps>
__global__ void __launch_bounds__(32 * (kWarps + kHelpers)) ttt_ssm_scan_kernel(const Params p, const int cblocks) {
    using Smem = ScanSmem<T>;
    constexpr int kTile = Smem::kTile, kQuads = Smem::kQuads, kPitch = Smem::kPitch, kNp = kWarps * kStates;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const Smem s(smem_raw, kWarps, kNp);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hid = tid - 32 * kWarps, helper = warp - kWarps;  // of the helpers
    const int b = (int)(blockIdx.x / cblocks), c0 = (int)(blockIdx.x % cblocks) * 32, c = c0 + lane;
    const bool on = c < p.C;
    const int len = length_of(p.lengths, b, p.T);
    const T* u_rows = static_cast<const T*>(p.u) + (long long)b * p.T * p.ld_u + c0;
    const T* dt_rows = static_cast<const T*>(p.dt) + (long long)b * p.T * p.ld_dt + c0;
    const T* z_rows = static_cast<const T*>(p.z) + (long long)b * p.T * p.ld_z + c0;
    const T* b_rows = static_cast<const T*>(p.Bm) + (long long)b * p.T * p.ld_b;
    const T* c_rows = static_cast<const T*>(p.Cm) + (long long)b * p.T * p.ld_c;
    T* y_rows = static_cast<T*>(p.y) + (long long)b * p.T * p.C + c;
    const int n0 = warp * kStates;

    // raw rows of tile m on their way
    const auto stage = [&](int m) {
        const int t0 = m * kTile, buf = m & 3, width = p.C - c0;
        stage_rows<T>(p.vec_rows, s.u + buf * kTile * 32, u_rows, p.ld_u, t0, kTile, len, 32, width, hid, 32 * kHelpers);
        stage_rows<T>(p.vec_rows, s.raw + buf * kTile * 32, dt_rows, p.ld_dt, t0, kTile, len, 32, width, hid, 32 * kHelpers);
        if (p.z) stage_rows<T>(p.vec_rows, s.z + buf * kTile * 32, z_rows, p.ld_z, t0, kTile, len, 32, width, hid, 32 * kHelpers);
        stage_rows<T>(p.vec_bc, s.rb + buf * kTile * kNp, b_rows, p.ld_b, t0, kTile, len, kNp, p.N, hid, 32 * kHelpers);
        stage_rows<T>(p.vec_bc, s.rc + buf * kTile * kNp, c_rows, p.ld_c, t0, kTile, len, kNp, p.N, hid, 32 * kHelpers);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f, skip = on && p.D ? p.D[c] : 0.f;
    // steps, inputs, B and C of tile m
    const auto prepare = [&](int m) {
        const int t0 = m * kTile, buf = m & 3, wb = m & 1;
        for (int q = helper; q < kQuads; q += kHelpers) {
            float dt[4], du[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int i = (buf * kTile + 4 * q + k) * 32 + lane;
                float d = to_f32(s.raw[i]) + bias;
                if (p.softplus) d = ssm::softplus(d);
                dt[k] = t0 + 4 * q + k < len ? d : 0.f;
                du[k] = dt[k] * to_f32(s.u[i]);
            }
            s.dt[(wb * kQuads + q) * 32 + lane] = make_float4(dt[0], dt[1], dt[2], dt[3]);
            s.du[(wb * kQuads + q) * 32 + lane] = make_float4(du[0], du[1], du[2], du[3]);
        }
        for (int i = hid; i < kTile * kNp; i += 32 * kHelpers) {
            const int at = (wb * kNp + i % kNp) * kPitch + i / kNp;
            s.b[at] = to_f32(s.rb[buf * kTile * kNp + i]);
            s.c[at] = to_f32(s.rc[buf * kTile * kNp + i]);
        }
    };
    // outputs of tile m: the sum over the warps, D and the gate
    const auto finish = [&](int m) {
        const int t0 = m * kTile, buf = m & 3, wb = m & 1;
        for (int q = helper; q < kQuads; q += kHelpers) {
            float4 y = s.y[(wb * kWarps * kQuads + q) * 32 + lane];
#pragma unroll
            for (int w = 1; w < kWarps; w++) {
                const float4 v = s.y[((wb * kWarps + w) * kQuads + q) * 32 + lane];
                y.x += v.x;
                y.y += v.y;
                y.z += v.z;
                y.w += v.w;
            }
            const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int i = (buf * kTile + 4 * q + k) * 32 + lane, t = t0 + 4 * q + k;
                float o[1] = {fmaf(skip, to_f32(s.u[i]), v[k])};
                if (p.z) {
                    const float z = to_f32(s.z[i]);
                    o[0] *= z * sigmoid(z);
                }
                if (on && t < len) store_vec<1>(y_rows + (long long)t * p.C, o);
            }
        }
    };

    float a2[kStates], h[kStates];
#pragma unroll
    for (int i = 0; i < kStates; i++) {
        const bool live = on && n0 + i < p.N && warp < kWarps;
        a2[i] = live ? rate(p.A[(size_t)c * p.N + n0 + i]) : 0.f;
        h[i] = live && p.h0 ? p.h0[((size_t)b * p.C + c) * p.N + n0 + i] : 0.f;
    }
    // the recursion over tile m
    const bool grows = warp_grows(p.softplus, a2);
    const auto walk = [&](int m, auto grow) {
        const int buf = m & 1;
        constexpr int kAt = 4;  // quads in work at once
        for (int q0 = 0; q0 < kQuads; q0 += kAt) {
            f2 dt[2 * kAt], du[2 * kAt], y[2 * kAt];
#pragma unroll
            for (int q = 0; q < kAt; q++) {
                const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&s.dt[(buf * kQuads + q0 + q) * 32 + lane]);
                const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(&s.du[(buf * kQuads + q0 + q) * 32 + lane]);
                dt[2 * q] = d.x;
                dt[2 * q + 1] = d.y;
                du[2 * q] = e.x;
                du[2 * q + 1] = e.y;
            }
#pragma unroll
            for (int i = 0; i < kStates; i++) {
                const f2 A2 = pack2(a2[i], a2[i]);
                f2 x[2 * kAt];
                float a[4 * kAt];
#pragma unroll
                for (int k = 0; k < 2 * kAt; k++) x[k] = mul2(dt[k], A2);
                decays<decltype(grow)::value>(a, x);
                const ulonglong2* Bi = reinterpret_cast<const ulonglong2*>(&s.b[(buf * kNp + n0 + i) * kPitch + 4 * q0]);
                const ulonglong2* Ci = reinterpret_cast<const ulonglong2*>(&s.c[(buf * kNp + n0 + i) * kPitch + 4 * q0]);
#pragma unroll
                for (int q = 0; q < kAt; q++) {
                    const ulonglong2 Bq = Bi[q], Cq = Ci[q];
                    const f2 in[2] = {mul2(du[2 * q], Bq.x), mul2(du[2 * q + 1], Bq.y)}, out[2] = {Cq.x, Cq.y};
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float lo, hi;
                        unpack2(in[k], lo, hi);
                        lo = fmaf(a[4 * q + 2 * k], h[i], lo);
                        h[i] = hi = fmaf(a[4 * q + 2 * k + 1], lo, hi);
                        y[2 * q + k] = i == 0 ? mul2(out[k], pack2(lo, hi)) : fma2(out[k], pack2(lo, hi), y[2 * q + k]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kAt; q++)
                *reinterpret_cast<ulonglong2*>(&s.y[((buf * kWarps + warp) * kQuads + q0 + q) * 32 + lane]) = make_ulonglong2(y[2 * q], y[2 * q + 1]);
        }
    };
    const int tiles = (len + kTile - 1) / kTile;
    // all but the newest of the copies have come in, for all helpers
    const auto arrived = [&](bool newest_too) {
        if (newest_too)
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        asm volatile("bar.sync 1, %0;" ::"r"(32 * kHelpers) : "memory");
    };
    if (warp >= kWarps && tiles > 0) {
        stage(0);
        if (tiles > 1) stage(1);
        arrived(tiles == 1);
        prepare(0);
    }
    __syncthreads();
    for (int m = 0; m <= tiles; m++) {
        if (warp >= kWarps) {
            if (m + 2 < tiles) stage(m + 2);
            if (m >= 1) finish(m - 1);
            if (m + 1 < tiles) {
                arrived(m + 2 >= tiles);
                prepare(m + 1);
            }
        } else if (m < tiles) {
            grows ? walk(m, std::true_type{}) : walk(m, std::false_type{});
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kStates; i++)
        if (on && warp < kWarps && n0 + i < p.N) p.h_T[((size_t)b * p.C + c) * p.N + n0 + i] = h[i];
    const float zero[1] = {0.f};
    for (int t = len + warp; t < p.T; t += kWarps + kHelpers)
        if (on) store_vec<1>(y_rows + (long long)t * p.C, zero);
}

template <typename T, int kWarps>
cudaError_t launch(const SsmArgs& a, cudaStream_t stream) {
    const Params p = params_of(a);
    const long long cblocks = (a.C + 31) / 32, grid = a.B * cblocks;
    if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
    const size_t smem = ScanSmem<T>::bytes(kWarps, kWarps * kStates);
    static_assert(ScanSmem<T>::bytes(4, 16) <= kMaxSmem, "fits an SM");
    const auto kernel = ttt_ssm_scan_kernel<T, kWarps>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)grid, 32 * (kWarps + kHelpers), smem, stream>>>(p, (int)cblocks);
    return cudaPeekAtLastError();
}

template <typename T>
cudaError_t launch_by_states(const SsmArgs& a, cudaStream_t stream) {
    if (a.N <= 4) return launch<T, 1>(a, stream);
    if (a.N <= 8) return launch<T, 2>(a, stream);
    return launch<T, 4>(a, stream);
}

}  // namespace

cudaError_t launch_ssm_scan(const SsmArgs& a, cudaStream_t stream) {
    if (a.N > 16) return cudaErrorInvalidValue;
    return a.dtype == TTT_BF16 ? launch_by_states<__nv_bfloat16>(a, stream) : launch_by_states<float>(a, stream);
}

}  // namespace ttt
