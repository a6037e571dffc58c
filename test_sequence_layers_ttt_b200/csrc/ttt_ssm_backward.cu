// Gradient of the selective state space scan.
//
// With dy' = dy silu(z) the gradient that reaches the scan's own output, and a_t = e^(dt_t A):
//   g_t = C_t dy'_t + a_{t+1} g_{t+1}          (g_T + the final state's gradient)
//   dC_t = sum over channels of dy'_t h_t,  dB_t = sum over channels of g_t dt_t u_t
//   du_t = dt_t (g_t . B_t) + D dy'_t,  ddt_t = (u_t (g_t . B_t) + sum_n g_t a_t h_{t-1} A) dt'(raw)
//   dA = sum_t g_t a_t h_{t-1} dt_t,  dD = sum_t dy'_t u_t,  dz_t = dy_t silu'(z_t) (C_t . h_t + D u_t)
//
// Two passes.  The first runs the scan and writes the state at the start of every chunk of kK tokens;
// the second takes the chunks from the last to the first: it recomputes a chunk's decays into registers and its
// states into shared memory and then walks it backwards.  A warp's lanes are 32 channels and a thread holds four states
// of one, so that B and C are one broadcast read each; the warps of a block share out the states.  Sums
// over states meet in shared memory, sums over the block's channels in shuffles; what is summed over
// blocks or sequences goes through the workspace and is added up in an order that the shape fixes.
// Where B and the channels make few blocks, the time axis is split too (split_of): one more pass takes each part
// for itself and leaves its end state, its gradient to the part before and its decay, from which the blocks of
// the two passes above fold the state and the gradient that they start from.
//
// Sums over tokens are of chunks' sums in fp32, added in 64 bits.  What is left of dA's error (4e-7 to 9e-7 of its
// norm over thousands of tokens) is the decays' rounding to fp32, which alone gives 4e-7 to 7e-7.
//
// Measured (8 x 2048 x 1536, 16 states): 1.02 ms in bf16, the second pass 0.80 and the first 0.22, and 1.01 in fp32.  The
// special functions would take 0.17 of it, HBM 0.05 for the inputs and outputs and 0.06 for the chunks' states and the
// blocks' parts of dB and dC, 100 MB each, written and read.  The second pass issues in 56 % of the clocks and keeps the
// shared memory pipe 60 % busy, most of it the shuffles and the states' way through shared memory.
#include "ssm_params.cuh"

#include <algorithm>
#include <type_traits>

namespace ttt {
namespace {

using namespace ssm;

struct SsmBwdParams {
    int B, T, C, N, chunks, cblocks;
    int segs, seg_len;  // parts of the time axis and their tokens
    long long ld_u, ld_dt, ld_b, ld_c, ld_z;
    int softplus;
    const void *u, *dt, *Bm, *Cm, *z, *dy;
    const float *dt_bias, *A, *D, *h0, *dh_T;
    const int* lengths;
    void *du, *ddt, *dz;
    float* dh0;
    float* ckpt;     // [B][chunks][4 kNW][C]
    float* part_bc;  // [cblocks][B][T][2][N]
    float* part_c;   // [B][segs][N + 2][C]: dA, dD, ddt_bias
    float* carry;    // [B][segs][4][4 kNW][C]: a part's end state from zero, its gradient to the part before, its decay in two factors
    bool vec_rows, vec_bc;
};

// The block's 32 channels and its part of a sequence: tokens t0 .. t0 + T, the first len of them no padding
struct Where {
    int b, seg, cblk, c0, t0, T, len;
};
__device__ __forceinline__ Where where(const SsmBwdParams& p) {
    Where w;
    const int row = (int)(blockIdx.x / p.cblocks);
    w.cblk = (int)(blockIdx.x % p.cblocks);
    w.c0 = w.cblk * 32;
    w.b = row / p.segs;
    w.seg = row % p.segs;
    w.t0 = w.seg * p.seg_len;
    w.T = min(p.T - w.t0, p.seg_len);
    w.len = max(min(length_of(p.lengths, w.b, p.T) - w.t0, w.T), 0);
    return w;
}
// Carry value m (0: state, 1: gradient, 2 and 3: the decay's factors) of part seg, of the thread's first state n0 and channel c
template <int kNp>
__device__ __forceinline__ size_t carry_at(const SsmBwdParams& p, int b, int seg, int m, int n0, int c) {
    return ((((size_t)b * p.segs + seg) * 4 + m) * kNp + n0) * p.C + c;
}
// v folded over `count` parts from part `from` on, in steps of `by`; m as in carry_at.  Eight parts' values are on
// their way at a time (four where a thread has 128 registers): one by one, 64 parts took longer than a walk along one of them.
template <int kNp, bool kGrow>
__device__ __forceinline__ void fold(float (&v)[kStates], const SsmBwdParams& p, int b, int from, int by, int count, int m,
                                     int n0, int c) {
    constexpr int kBatch = kNp > 16 ? 4 : 8;
    for (int j0 = 0; j0 < count; j0 += kBatch) {
        float e[kBatch][kStates], a0[kBatch][kStates], a1[kBatch][kStates];
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
            const bool live = j0 + j < count;
            const int seg = live ? from + (j0 + j) * by : 0;
            const float *pe = p.carry + carry_at<kNp>(p, b, seg, m, n0, c), *p0 = p.carry + carry_at<kNp>(p, b, seg, 2, n0, c);
            const float* p1 = p.carry + carry_at<kNp>(p, b, seg, 3, n0, c);  // 1 where no state of the warp grows
#pragma unroll
            for (int i = 0; i < kStates; i++) {
                e[j][i] = live ? pe[(size_t)i * p.C] : 0.f;
                a0[j][i] = live ? p0[(size_t)i * p.C] : 1.f;
                a1[j][i] = kGrow && live ? p1[(size_t)i * p.C] : 1.f;
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; j++)
#pragma unroll
            for (int i = 0; i < kStates; i++) v[i] = kGrow ? carried(v[i], a0[j][i], a1[j][i], e[j][i]) : fmaf(a0[j][i], v[i], e[j][i]);
    }
}

// Rows of a tile of kK tokens as they come from memory
template <typename T, int kK, int kNp>
struct RawTile {
    T u[kK][32], dt[kK][32], z[kK][32], dy[kK][32];
    T b[kK][kNp], c[kK][kNp];
};

// ---------------------------------------------------------------- pass 1: the states at the chunks' starts
template <typename T, int kNW, int kTile, bool kEnds>
struct CkptSmem {
    RawTile<T, kTile, kStates * kNW> raw[2];
    float4 dt[kTile / 4][32], du[kTile / 4][32], dy[kEnds ? kTile / 4 : 1][32];
    float b[kStates * kNW][kTile + 4], c[kEnds ? kStates * kNW : 1][kTile + 4];
};

// kK: tokens of a chunk; a tile is two chunks.  kEnds: a part of the time axis for itself, as carry has it.
// The gradient that leaves a part to the one before is sum_t (a_first ... a_t) C_t dy'_t, so it too is
// summed walking forwards; of states that grow the product of the even tokens' decays and that of the odd ones' are kept
// apart, as carried() takes them.
template <typename T, int kNW, int kK, bool kEnds>
__global__ void __launch_bounds__(32 * kNW) ttt_ssm_checkpoint_kernel(const SsmBwdParams p) {
    constexpr int kNp = kStates * kNW, kTile = 2 * kK, kThreads = 32 * kNW;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    CkptSmem<T, kNW, kTile, kEnds>& s = *reinterpret_cast<CkptSmem<T, kNW, kTile, kEnds>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Where w = where(p);
    const int c = w.c0 + lane;
    const bool on = c < p.C;
    const int len = w.len;
    const int n_chunks = (len + kK - 1) / kK, tiles = (len + kTile - 1) / kTile;
    const int n0 = warp * kStates;
    float h[kStates], a2[kStates], back[kStates], all[2][kStates];
#pragma unroll
    for (int i = 0; i < kStates; i++) {
        const bool live = on && n0 + i < p.N;
        a2[i] = live ? rate(p.A[(size_t)c * p.N + n0 + i]) : 0.f;
        h[i] = !kEnds && live && p.h0 ? p.h0[((size_t)w.b * p.C + c) * p.N + n0 + i] : 0.f;
        back[i] = 0.f;
        all[0][i] = all[1][i] = 1.f;
    }
    const bool grows = warp_grows(p.softplus, a2);
    if (!kEnds && on) {
        if (grows)
            fold<kNp, true>(h, p, w.b, 0, 1, w.seg, 0, n0, c);
        else
            fold<kNp, false>(h, p, w.b, 0, 1, w.seg, 0, n0, c);
    }
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f;
    const long long row0 = (long long)w.b * p.T + w.t0;
    const auto stage = [&](int m) {
        RawTile<T, kTile, kNp>& r = s.raw[m & 1];
        const int t0 = m * kTile, width = p.C - w.c0;
        stage_rows<T>(p.vec_rows, &r.u[0][0], static_cast<const T*>(p.u) + row0 * p.ld_u + w.c0, p.ld_u, t0, kTile, len, 32, width, tid, kThreads);
        stage_rows<T>(p.vec_rows, &r.dt[0][0], static_cast<const T*>(p.dt) + row0 * p.ld_dt + w.c0, p.ld_dt, t0, kTile, len, 32, width, tid, kThreads);
        stage_rows<T>(p.vec_bc, &r.b[0][0], static_cast<const T*>(p.Bm) + row0 * p.ld_b, p.ld_b, t0, kTile, len, kNp, p.N, tid, kThreads);
        if (kEnds) {
            stage_rows<T>(p.vec_rows, &r.dy[0][0], static_cast<const T*>(p.dy) + row0 * p.C + w.c0, p.C, t0, kTile, len, 32, width, tid, kThreads);
            if (p.z)
                stage_rows<T>(p.vec_rows, &r.z[0][0], static_cast<const T*>(p.z) + row0 * p.ld_z + w.c0, p.ld_z, t0, kTile, len, 32, width, tid, kThreads);
            stage_rows<T>(p.vec_bc, &r.c[0][0], static_cast<const T*>(p.Cm) + row0 * p.ld_c, p.ld_c, t0, kTile, len, kNp, p.N, tid, kThreads);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (tiles > 0) stage(0);
    for (int m = 0; m < tiles; m++) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (m + 1 < tiles) stage(m + 1);
        const RawTile<T, kTile, kNp>& r = s.raw[m & 1];
        for (int q = warp; q < kTile / 4; q += kNW) {
            float dt[4], du[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const float raw = to_f32(r.dt[4 * q + k][lane]) + bias;
                dt[k] = m * kTile + 4 * q + k < len ? (p.softplus ? ssm::softplus(raw) : raw) : 0.f;
                du[k] = dt[k] * to_f32(r.u[4 * q + k][lane]);
            }
            s.dt[q][lane] = make_float4(dt[0], dt[1], dt[2], dt[3]);
            s.du[q][lane] = make_float4(du[0], du[1], du[2], du[3]);
            if constexpr (kEnds) {
                float dy[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    dy[k] = to_f32(r.dy[4 * q + k][lane]);
                    if (p.z) {
                        const float z = to_f32(r.z[4 * q + k][lane]);
                        dy[k] *= z * sigmoid(z);
                    }
                }
                s.dy[q][lane] = make_float4(dy[0], dy[1], dy[2], dy[3]);
            }
        }
        for (int i = tid; i < kTile * kNp; i += kThreads) {
            s.b[i % kNp][i / kNp] = to_f32(r.b[i / kNp][i % kNp]);
            if constexpr (kEnds) s.c[i % kNp][i / kNp] = to_f32(r.c[i / kNp][i % kNp]);
        }
        __syncthreads();
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int chunk = 2 * m + half;
            if (!kEnds && on && chunk < n_chunks) {
                float* out = p.ckpt + (((size_t)w.b * p.chunks + w.t0 / kK + chunk) * kNp + n0) * p.C + c;
#pragma unroll
                for (int i = 0; i < kStates; i++) out[(size_t)i * p.C] = h[i];
            }
            constexpr int kQ = kK / 4;
            f2 dt[2 * kQ], du[2 * kQ], dy[2 * kQ];
#pragma unroll
            for (int q = 0; q < kQ; q++) {
                const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&s.dt[half * kQ + q][lane]);
                const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(&s.du[half * kQ + q][lane]);
                dt[2 * q] = d.x;
                dt[2 * q + 1] = d.y;
                du[2 * q] = e.x;
                du[2 * q + 1] = e.y;
                if constexpr (kEnds) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&s.dy[half * kQ + q][lane]);
                    dy[2 * q] = f.x;
                    dy[2 * q + 1] = f.y;
                }
            }
            const auto walk = [&](auto grow) {
#pragma unroll
                for (int i = 0; i < kStates; i++) {
                    const f2 A2 = pack2(a2[i], a2[i]);
                    f2 x[2 * kQ];
                    float a[4 * kQ];
#pragma unroll
                    for (int k = 0; k < 2 * kQ; k++) x[k] = mul2(dt[k], A2);
                    decays<decltype(grow)::value>(a, x);
                    const ulonglong2* Bi = reinterpret_cast<const ulonglong2*>(&s.b[n0 + i][half * kK]);
#pragma unroll
                    for (int q = 0; q < kQ; q++) {
                        const ulonglong2 Bq = Bi[q];
                        float v0, v1, v2, v3;
                        unpack2(mul2(du[2 * q], Bq.x), v0, v1);
                        unpack2(mul2(du[2 * q + 1], Bq.y), v2, v3);
                        h[i] = fmaf(a[4 * q], h[i], v0);
                        h[i] = fmaf(a[4 * q + 1], h[i], v1);
                        h[i] = fmaf(a[4 * q + 2], h[i], v2);
                        h[i] = fmaf(a[4 * q + 3], h[i], v3);
                        if constexpr (kEnds) {
                            const ulonglong2 Cq = reinterpret_cast<const ulonglong2*>(&s.c[n0 + i][half * kK])[q];
                            float g[4];
                            unpack2(mul2(dy[2 * q], Cq.x), g[0], g[1]);
                            unpack2(mul2(dy[2 * q + 1], Cq.y), g[2], g[3]);
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                if constexpr (decltype(grow)::value) {
                                    all[k & 1][i] *= a[4 * q + k];
                                    back[i] = carried(g[k], all[0][i], all[1][i], back[i]);
                                } else {
                                    all[0][i] *= a[4 * q + k];
                                    back[i] = fmaf(all[0][i], g[k], back[i]);
                                }
                            }
                        }
                    }
                }
            };
            grows ? walk(std::true_type{}) : walk(std::false_type{});
        }
    }
    if (kEnds && on) {
#pragma unroll
        for (int i = 0; i < kStates; i++) {
            p.carry[carry_at<kNp>(p, w.b, w.seg, 0, n0 + i, c)] = h[i];
            p.carry[carry_at<kNp>(p, w.b, w.seg, 1, n0 + i, c)] = back[i];
            p.carry[carry_at<kNp>(p, w.b, w.seg, 2, n0 + i, c)] = all[0][i];
            p.carry[carry_at<kNp>(p, w.b, w.seg, 3, n0 + i, c)] = all[1][i];
        }
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

template <typename T, int kNW, int kK>
struct BwdSmem {
    RawTile<T, kK, kStates * kNW> raw[2];
    float b[kStates * kNW][kK + 4], c[kStates * kNW][kK + 4];
    float4 dt[kK / 4][32], du[kK / 4][32], dy[kK / 4][32];  // dt, dt u, dy'
    float4 slope[kK / 4][32], dyz[kK / 4][32];              // d dt / d raw, dy silu'(z)
    // a thread's states after each token, four tokens of a state together; once a quad has been walked back, its
    // first three places hold the thread's parts of g . B, of the sum with A, and of C . h
    float4 h[kK / 4][kStates][32 * kNW];
    // sums over all tokens, of chunks' sums in fp32: their terms cancel, and a thousand roundings of one fp32 sum would
    // show in the result
    double dA[kStates][32 * kNW], sum[kNW][2][32];
};
// Blocks an SM of the second pass: 384 threads with 168 registers each (the decays of a chunk are 64 of them),
// where keeping the states there too left room for 256.
constexpr int blocks_for(int kNW) { return kNW >= 8 ? 1 : 12 / kNW; }

template <typename T, int kNW, int kK>
__global__ void __launch_bounds__(32 * kNW, blocks_for(kNW)) ttt_ssm_backward_kernel(const SsmBwdParams p) {
    constexpr int kNp = kStates * kNW, kQ = kK / 4, kThreads = 32 * kNW;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<T, kNW, kK>& s = *reinterpret_cast<BwdSmem<T, kNW, kK>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Where w = where(p);
    const int c = w.c0 + lane;
    const bool on = c < p.C;
    const int len = w.len;
    const int n_chunks = (len + kK - 1) / kK;
    const int n0 = warp * kStates;
    const long long row0 = (long long)w.b * p.T + w.t0;
    float a2[kStates], g[kStates], first[kStates];
#pragma unroll
    for (int i = 0; i < kStates; i++) {
        const bool live = on && n0 + i < p.N;
        a2[i] = live ? rate(p.A[(size_t)c * p.N + n0 + i]) : 0.f;
        g[i] = live && p.dh_T ? p.dh_T[((size_t)w.b * p.C + c) * p.N + n0 + i] : 0.f;
        s.dA[i][tid] = 0.0;
    }
    if (warp_grows(p.softplus, a2)) {
        if (on) fold<kNp, true>(g, p, w.b, p.segs - 1, -1, p.segs - 1 - w.seg, 1, n0, c);
    } else if (on) {
        fold<kNp, false>(g, p, w.b, p.segs - 1, -1, p.segs - 1 - w.seg, 1, n0, c);
    }
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f, skip = on && p.D ? p.D[c] : 0.f;
    double dD = 0.0, dbias = 0.0;

    // rows of padding: zero gradients
    for (int t = len + warp; t < w.T; t += kNW) {
        if (on) {
            const size_t at = ((size_t)row0 + t) * p.C + c;
            const float zero[1] = {0.f};
            store_vec<1>(static_cast<T*>(p.du) + at, zero);
            store_vec<1>(static_cast<T*>(p.ddt) + at, zero);
            if (p.dz) store_vec<1>(static_cast<T*>(p.dz) + at, zero);
        }
    }

    const auto stage = [&](int chunk) {
        RawTile<T, kK, kNp>& r = s.raw[chunk & 1];
        const int t0 = chunk * kK, width = p.C - w.c0;
        stage_rows<T>(p.vec_rows, &r.u[0][0], static_cast<const T*>(p.u) + row0 * p.ld_u + w.c0, p.ld_u, t0, kK, len, 32, width, tid, kThreads);
        stage_rows<T>(p.vec_rows, &r.dt[0][0], static_cast<const T*>(p.dt) + row0 * p.ld_dt + w.c0, p.ld_dt, t0, kK, len, 32, width, tid, kThreads);
        stage_rows<T>(p.vec_rows, &r.dy[0][0], static_cast<const T*>(p.dy) + row0 * p.C + w.c0, p.C, t0, kK, len, 32, width, tid, kThreads);
        if (p.z)
            stage_rows<T>(p.vec_rows, &r.z[0][0], static_cast<const T*>(p.z) + row0 * p.ld_z + w.c0, p.ld_z, t0, kK, len, 32, width, tid, kThreads);
        stage_rows<T>(p.vec_bc, &r.b[0][0], static_cast<const T*>(p.Bm) + row0 * p.ld_b, p.ld_b, t0, kK, len, kNp, p.N, tid, kThreads);
        stage_rows<T>(p.vec_bc, &r.c[0][0], static_cast<const T*>(p.Cm) + row0 * p.ld_c, p.ld_c, t0, kK, len, kNp, p.N, tid, kThreads);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto load_first = [&](int chunk) {
        const float* in = p.ckpt + (((size_t)w.b * p.chunks + w.t0 / kK + chunk) * kNp + n0) * p.C + c;
#pragma unroll
        for (int i = 0; i < kStates; i++) first[i] = on ? in[(size_t)i * p.C] : 0.f;
    };
    if (n_chunks > 0) {
        stage(n_chunks - 1);
        load_first(n_chunks - 1);
    }
    for (int chunk = n_chunks - 1; chunk >= 0; chunk--) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (chunk > 0) stage(chunk - 1);
        const RawTile<T, kK, kNp>& r = s.raw[chunk & 1];
        for (int q = warp; q < kQ; q += kNW) {
            float dt[4], du[4], dy[4], slope[4], dyz[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int j = 4 * q + k;
                const bool live = chunk * kK + j < len;
                const float raw = to_f32(r.dt[j][lane]) + bias;
                dt[k] = live ? (p.softplus ? ssm::softplus(raw) : raw) : 0.f;
                slope[k] = p.softplus ? sigmoid(raw) : 1.f;
                du[k] = dt[k] * to_f32(r.u[j][lane]);
                dy[k] = to_f32(r.dy[j][lane]);
                dyz[k] = 0.f;
                if (p.z) {
                    const float z = to_f32(r.z[j][lane]), sg = sigmoid(z);
                    dyz[k] = dy[k] * sg * (1.f + z * (1.f - sg));
                    dy[k] *= z * sg;
                }
            }
            s.dt[q][lane] = make_float4(dt[0], dt[1], dt[2], dt[3]);
            s.du[q][lane] = make_float4(du[0], du[1], du[2], du[3]);
            s.dy[q][lane] = make_float4(dy[0], dy[1], dy[2], dy[3]);
            s.slope[q][lane] = make_float4(slope[0], slope[1], slope[2], slope[3]);
            s.dyz[q][lane] = make_float4(dyz[0], dyz[1], dyz[2], dyz[3]);
        }
        for (int i = tid; i < kK * kNp; i += kThreads) {
            s.b[i % kNp][i / kNp] = to_f32(r.b[i / kNp][i % kNp]);
            s.c[i % kNp][i / kNp] = to_f32(r.c[i / kNp][i % kNp]);
        }
        __syncthreads();
        float a[kStates][kK], start[kStates];
        {
            f2 dt[2 * kQ], du[2 * kQ];
#pragma unroll
            for (int q = 0; q < kQ; q++) {
                const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&s.dt[q][lane]);
                const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(&s.du[q][lane]);
                dt[2 * q] = d.x;
                dt[2 * q + 1] = d.y;
                du[2 * q] = e.x;
                du[2 * q + 1] = e.y;
            }
#pragma unroll
            for (int i = 0; i < kStates; i++) {
                const f2 A2 = pack2(a2[i], a2[i]);
                f2 x[2 * kQ];
#pragma unroll
                for (int k = 0; k < 2 * kQ; k++) x[k] = mul2(dt[k], A2);
                decays<true>(a[i], x);
                const ulonglong2* Bi = reinterpret_cast<const ulonglong2*>(&s.b[n0 + i][0]);
                float h = start[i] = first[i];
#pragma unroll
                for (int q = 0; q < kQ; q++) {
                    const ulonglong2 Bq = Bi[q];
                    float v[4];
                    unpack2(mul2(du[2 * q], Bq.x), v[0], v[1]);
                    unpack2(mul2(du[2 * q + 1], Bq.y), v[2], v[3]);
#pragma unroll
                    for (int k = 0; k < 4; k++) v[k] = h = fmaf(a[i][4 * q + k], h, v[k]);
                    s.h[q][i][tid] = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        if (chunk > 0) load_first(chunk - 1);
        float dA[kStates] = {};
#pragma unroll
        for (int q = kQ - 1; q >= 0; q--) {
            asm volatile("" ::: "memory");  // the loads of one quad at a time: hoisted together they spill
            float v[32];  // of four tokens: dB and dC of the thread's four states
            const ulonglong2 dt = *reinterpret_cast<const ulonglong2*>(&s.dt[q][lane]);
            const ulonglong2 du = *reinterpret_cast<const ulonglong2*>(&s.du[q][lane]);
            const ulonglong2 dy = *reinterpret_cast<const ulonglong2*>(&s.dy[q][lane]);
            float d[4];
            unpack2(dy.x, d[0], d[1]);
            unpack2(dy.y, d[2], d[3]);
            f2 gb[2], ga[2], y[2];
#pragma unroll
            for (int i = 0; i < kStates; i++) {
                const ulonglong2 Bq = *reinterpret_cast<const ulonglong2*>(&s.b[n0 + i][4 * q]);
                const ulonglong2 Cq = *reinterpret_cast<const ulonglong2*>(&s.c[n0 + i][4 * q]);
                const float4 after = s.h[q][i][tid];
                const float before[4] = {q > 0 ? s.h[(q + kQ - 1) % kQ][i][tid].w : start[i], after.x, after.y, after.z};
                float ct[4], gk[4], x[4];
                unpack2(Cq.x, ct[0], ct[1]);
                unpack2(Cq.y, ct[2], ct[3]);
#pragma unroll
                for (int k = 3; k >= 0; k--) {
                    gk[k] = fmaf(ct[k], d[k], g[i]);
                    g[i] = gk[k] * a[i][4 * q + k];
                    x[k] = g[i] * before[k];
                }
                const f2 g0 = pack2(gk[0], gk[1]), g1 = pack2(gk[2], gk[3]);
                const f2 h0 = pack2(after.x, after.y), h1 = pack2(after.z, after.w);
                const f2 x0 = pack2(x[0], x[1]), x1 = pack2(x[2], x[3]), A2 = pack2(a2[i], a2[i]);
                unpack2(mul2(g0, du.x), v[i], v[8 + i]);
                unpack2(mul2(g1, du.y), v[16 + i], v[24 + i]);
                unpack2(mul2(dy.x, h0), v[4 + i], v[12 + i]);
                unpack2(mul2(dy.y, h1), v[20 + i], v[28 + i]);
                gb[0] = i == 0 ? mul2(g0, Bq.x) : fma2(g0, Bq.x, gb[0]);
                gb[1] = i == 0 ? mul2(g1, Bq.y) : fma2(g1, Bq.y, gb[1]);
                y[0] = i == 0 ? mul2(h0, Cq.x) : fma2(h0, Cq.x, y[0]);
                y[1] = i == 0 ? mul2(h1, Cq.y) : fma2(h1, Cq.y, y[1]);
                ga[0] = i == 0 ? mul2(x0, A2) : fma2(x0, A2, ga[0]);
                ga[1] = i == 0 ? mul2(x1, A2) : fma2(x1, A2, ga[1]);
                float lo, hi;
                unpack2(fma2(x1, dt.y, mul2(x0, dt.x)), lo, hi);
                dA[i] += lo + hi;
            }
            *reinterpret_cast<ulonglong2*>(&s.h[q][0][tid]) = make_ulonglong2(gb[0], gb[1]);
            *reinterpret_cast<ulonglong2*>(&s.h[q][1][tid]) = make_ulonglong2(ga[0], ga[1]);
            *reinterpret_cast<ulonglong2*>(&s.h[q][2][tid]) = make_ulonglong2(y[0], y[1]);
            const float sum = sum_scatter(v, lane);
            const int t = chunk * kK + 4 * q + (lane >> 3), n = n0 + (lane & 3);
            if (t < len && n < p.N)
                p.part_bc[((((size_t)w.cblk * p.B + w.b) * p.T + w.t0 + t) * 2 + ((lane >> 2) & 1)) * p.N + n] = sum;
        }
#pragma unroll
        for (int i = 0; i < kStates; i++) s.dA[i][tid] += dA[i];
        __syncthreads();
        for (int q = warp; q < kQ; q += kNW) {
            float sum_D = 0.f, sum_bias = 0.f;
            float4 gb = s.h[q][0][lane], ga = s.h[q][1][lane], y = s.h[q][2][lane];
#pragma unroll
            for (int k = 1; k < kNW; k++) {
                const int from = 32 * k + lane;
                const float4 b4 = s.h[q][0][from], a4 = s.h[q][1][from], y4 = s.h[q][2][from];
                gb = make_float4(gb.x + b4.x, gb.y + b4.y, gb.z + b4.z, gb.w + b4.w);
                ga = make_float4(ga.x + a4.x, ga.y + a4.y, ga.z + a4.z, ga.w + a4.w);
                y = make_float4(y.x + y4.x, y.y + y4.y, y.z + y4.z, y.w + y4.w);
            }
            const float4 dt4 = s.dt[q][lane], dy4 = s.dy[q][lane], sl4 = s.slope[q][lane], dz4 = s.dyz[q][lane];
            const float gbs[4] = {gb.x, gb.y, gb.z, gb.w}, gas[4] = {ga.x, ga.y, ga.z, ga.w}, ys[4] = {y.x, y.y, y.z, y.w};
            const float dts[4] = {dt4.x, dt4.y, dt4.z, dt4.w}, dys[4] = {dy4.x, dy4.y, dy4.z, dy4.w};
            const float sls[4] = {sl4.x, sl4.y, sl4.z, sl4.w}, dzs[4] = {dz4.x, dz4.y, dz4.z, dz4.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int t = chunk * kK + 4 * q + k;
                if (!on || t >= len) continue;
                const float u = to_f32(r.u[4 * q + k][lane]);
                const size_t at = ((size_t)row0 + t) * p.C + c;
                const float o_u[1] = {fmaf(dts[k], gbs[k], skip * dys[k])};
                const float o_dt[1] = {fmaf(u, gbs[k], gas[k] * (1.f / kLog2e)) * sls[k]};
                store_vec<1>(static_cast<T*>(p.du) + at, o_u);
                store_vec<1>(static_cast<T*>(p.ddt) + at, o_dt);
                if (p.dz) {
                    const float o_z[1] = {dzs[k] * fmaf(skip, u, ys[k])};
                    store_vec<1>(static_cast<T*>(p.dz) + at, o_z);
                }
                sum_D = fmaf(dys[k], u, sum_D);
                sum_bias += o_dt[0];
            }
            dD += sum_D;
            dbias += sum_bias;
        }
    }
    s.sum[warp][0][lane] = dD;
    s.sum[warp][1][lane] = dbias;
    __syncthreads();
    if (on) {
        const size_t row = (size_t)w.b * p.segs + w.seg;
#pragma unroll
        for (int i = 0; i < kStates; i++) {
            if (n0 + i < p.N) {
                p.part_c[(row * (p.N + 2) + n0 + i) * p.C + c] = (float)s.dA[i][tid];
                if (p.dh0 && w.seg == 0) p.dh0[((size_t)w.b * p.C + c) * p.N + n0 + i] = g[i];
            }
        }
        if (warp == 0) {
            double x = 0.0, y = 0.0;
#pragma unroll
            for (int q = 0; q < kNW; q++) {
                x += s.sum[q][0][lane];
                y += s.sum[q][1][lane];
            }
            p.part_c[(row * (p.N + 2) + p.N) * p.C + c] = (float)x;
            p.part_c[(row * (p.N + 2) + p.N + 1) * p.C + c] = (float)y;
        }
    }
}

// ---------------------------------------------------------------- the sums over blocks and sequences
struct SsmSums {
    int B, T, C, N, cblocks, rows;  // rows: parts of sequences
    unsigned bc_blocks;             // blocks that sum dB and dC; the others sum dA, dD and ddt_bias
    const int* lengths;
    const float *part_bc, *part_c;
    float *dB, *dC, *dA, *dD, *dbias;
};
__global__ void __launch_bounds__(256) ttt_ssm_sum_kernel(const SsmSums p) {
    __shared__ double sums[8][32];
    if (blockIdx.x < p.bc_blocks) {
        const size_t per = (size_t)p.T * 2 * p.N, total = (size_t)p.B * per;
        const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= total) return;
        const int b = (int)(i / per);
        const size_t r = i % per;
        const int t = (int)(r / (2 * p.N)), m = (int)(r % (2 * p.N));
        float a = 0.f;
        if (t < length_of(p.lengths, b, p.T))
            for (int k = 0; k < p.cblocks; k++) a += p.part_bc[(size_t)k * total + i];
        (m < p.N ? p.dB : p.dC)[((size_t)b * p.T + t) * p.N + (m < p.N ? m : m - p.N)] = a;
        return;
    }
    // 32 columns a block; its eight warps share out the rows
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t cols = (size_t)(p.N + 2) * p.C, i = (size_t)(blockIdx.x - p.bc_blocks) * 32 + lane;
    double a = 0.0;
    if (i < cols) {
#pragma unroll 4
        for (int r = warp; r < p.rows; r += 8) a += p.part_c[(size_t)r * cols + i];
    }
    sums[warp][lane] = a;
    __syncthreads();
    if (warp != 0 || i >= cols) return;
    for (int k = 1; k < 8; k++) a += sums[k][lane];
    const int n = (int)(i / p.C), c = (int)(i % p.C);
    if (n < p.N)
        p.dA[(size_t)c * p.N + n] = (float)a;
    else if (n == p.N) {
        if (p.dD) p.dD[c] = (float)a;
    } else if (p.dbias) {
        p.dbias[c] = (float)a;
    }
}

constexpr int warps_for(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
// 16 tokens a chunk keep 64 decays in registers; with 16 warps a thread has 128 registers in all, so 8 there
constexpr int chunk_for(int kNW) { return kNW <= 8 ? 16 : 8; }

// Parts of the time axis.  A launch of few blocks waits on its own results, some 600 clocks a token.  So where the blocks
// fill at most half of the places that the SMs have for them, the axis is split into as many parts as there are
// places for, whole tiles each and at most 64, which is what the walk over the parts' ends costs.  Measured, split
// against whole (bf16, 16 states, 444 places): 4 blocks of 2641 tokens 58 us against 898, 36 of 614 68 against 320,
// 128 of 1024 241 against 363, 192 of 1024 345 against 414.
struct Split {
    int segs, seg_len;
};
Split split_of(int B, int T, int C, int N) {
    const int nw = warps_for(N), tile = 2 * chunk_for(nw);
    const long long blocks = (long long)B * ((C + 31) / 32), places = 148LL * blocks_for(nw);
    const int tiles = (int)(((long long)T + tile - 1) / tile);
    if (2 * blocks > places || tiles < 2) return {1, tiles > 0 ? tiles * tile : tile};
    const long long want = std::min<long long>({places / blocks, tiles, 64});
    const int per = (int)((tiles + want - 1) / want);
    return {(tiles + per - 1) / per, per * tile};
}

struct Layout {
    size_t ckpt, part_bc, part_c, carry, total;  // floats
};
Layout layout(int B, int T, int C, int N) {
    const int nw = warps_for(N), K = chunk_for(nw);
    const size_t chunks = ((size_t)T + K - 1) / K, cblocks = ((size_t)C + 31) / 32;
    const auto up = [](size_t x) { return (x + 3) / 4 * 4; };
    Layout l{};
    l.ckpt = up((size_t)B * chunks * kStates * nw * C);
    l.part_bc = up(cblocks * B * T * 2 * N);
    const size_t segs = (size_t)split_of(B, T, C, N).segs;
    l.part_c = up(B * segs * (N + 2) * C);
    l.carry = segs > 1 ? up(B * segs * 4 * kStates * nw * C) : 0;
    l.total = l.ckpt + l.part_bc + l.part_c + l.carry;
    return l;
}

template <typename T, int kNW>
cudaError_t launch(const SsmBwdParams& p, cudaStream_t stream) {
    constexpr int kK = chunk_for(kNW);
    const unsigned grid = (unsigned)((long long)p.B * p.segs * p.cblocks);
    const auto ends = ttt_ssm_checkpoint_kernel<T, kNW, kK, true>;
    const auto first = ttt_ssm_checkpoint_kernel<T, kNW, kK, false>;
    const auto second = ttt_ssm_backward_kernel<T, kNW, kK>;
    constexpr int smem0 = (int)sizeof(CkptSmem<T, kNW, 2 * kK, true>), smem1 = (int)sizeof(CkptSmem<T, kNW, 2 * kK, false>);
    constexpr int smem2 = (int)sizeof(BwdSmem<T, kNW, kK>);
    static_assert(smem0 <= (int)kMaxSmem && smem1 <= (int)kMaxSmem && smem2 <= (int)kMaxSmem, "fits an SM");
    cudaError_t e = cudaFuncSetAttribute(first, cudaFuncAttributeMaxDynamicSharedMemorySize, smem1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(second, cudaFuncAttributeMaxDynamicSharedMemorySize, smem2);
    if (e == cudaSuccess && p.segs > 1) {
        e = cudaFuncSetAttribute(ends, cudaFuncAttributeMaxDynamicSharedMemorySize, smem0);
        if (e != cudaSuccess) return e;
        ends<<<grid, 32 * kNW, smem0, stream>>>(p);
        e = cudaPeekAtLastError();
    }
    if (e != cudaSuccess) return e;
    first<<<grid, 32 * kNW, smem1, stream>>>(p);
    e = cudaPeekAtLastError();
    if (e != cudaSuccess) return e;
    second<<<grid, 32 * kNW, smem2, stream>>>(p);
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
    const Split split = split_of(f.B, f.T, f.C, f.N);
    p.segs = split.segs;
    p.seg_len = split.seg_len;
    if ((long long)p.B * p.segs * p.cblocks >= (1LL << 31)) return cudaErrorInvalidValue;
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
    p.carry = p.part_c + l.part_c;
    const int es = f.dtype == TTT_BF16 ? 2 : 4;
    p.vec_rows = rows16(f.u, f.ld_u, f.C, es) && rows16(f.dt, f.ld_dt, f.C, es) && rows16(f.z, f.ld_z, f.C, es) &&
                 rows16(a.dy, f.C, f.C, es);
    p.vec_bc = rows16(f.Bm, f.ld_b, f.N, es) && rows16(f.Cm, f.ld_c, f.N, es);
    cudaError_t e = f.dtype == TTT_BF16 ? dispatch<__nv_bfloat16>(p, stream) : dispatch<float>(p, stream);
    if (e != cudaSuccess) return e;
    const size_t bc = ((size_t)f.B * f.T * 2 * f.N + 255) / 256, ch = ((size_t)(f.N + 2) * f.C + 31) / 32;
    if (bc + ch >= (1ULL << 31)) return cudaErrorInvalidValue;
    const SsmSums sums{f.B, f.T, f.C, f.N, p.cblocks, f.B * p.segs, (unsigned)bc, f.lengths,
                       p.part_bc, p.part_c, a.dB, a.dC, a.dA, a.dD, a.ddt_bias};
    ttt_ssm_sum_kernel<<<(unsigned)(bc + ch), 256, 0, stream>>>(sums);
    return cudaPeekAtLastError();
}

}  // namespace ttt
