// Selective scan with a tile's tokens shared out among the warps of a block.
//
// A block takes kL channels of one sequence, tile by tile; a warp takes kSeg tokens of the tile for all of
// them, with kQ = 32 / kL lanes a channel sharing out the states in fours.  Per four states a thread
// computes its tokens' decays and inputs into registers and runs them from zero; the ends and the decays
// over the whole segments go through shared memory, every warp folds those before its own onto the tile's
// first state, and runs its tokens again from there.  The special functions are evaluated once a token and
// state all the same, and a channel keeps eight warps' worth of independent tokens in flight, which is what
// a launch of few channels needs: a token takes 61 clocks for 8 channels of 16 states (bf16), where a
// recursion that walks one token at a time takes 75 and more.  Measured: 5 x 3001 x 203 in fp32 107 us; the eight warps
// go through staging, conversion, both walks and the exchange in step, and a scheduler issues in 37 % of the clocks.
// 2 x 4096 x 2048 channels of 64 states, 32 channels a block, 0.84 ms (bf16).  Where even so most SMs have no block,
// the blocks of a cluster share out the tokens of one sequence the same way, through each other's shared memory (kSplit).
#include "ssm_params.cuh"

#include <cooperative_groups.h>
#include <type_traits>

namespace ttt {
namespace {

using namespace ssm;
namespace cg = cooperative_groups;

constexpr int kSeg = 16;      // tokens a warp takes of a tile
constexpr int kMaxWarps = 8;  // 128 tokens a tile; a thread's 64 decays and 64 inputs take 250 registers

// Shared memory, for tiles of `tile` tokens: raw rows of the tile in work and of the next one,
// B and C as floats, A log2(e), the state that goes from tile to tile, the segments' ends and decays.
template <typename T, int kL>
struct SegSmem {
    float4 *end, *fall;  // [2][kMaxWarps][32]; fall: the decays or their roots
    float4 *a2, *h;      // [groups][32]; [2][groups][32]
    float *b, *c;        // [n_pad][tile + 4]: a state's tokens side by side
    T *u, *dt, *z;       // [2][tile][kL]
    T *rb, *rc;          // [2][tile][n_pad]

    __host__ __device__ static size_t bytes(int tile, int n_pad) {
        const size_t groups = n_pad / (kStates * (32 / kL));
        return (4 * kMaxWarps + 3 * groups) * 32 * sizeof(float4) + 2 * n_pad * (size_t)(tile + 4) * sizeof(float) +
               (size_t)tile * (4 * n_pad + 6 * kL) * sizeof(T);
    }
    __device__ SegSmem(unsigned char* raw, int tile, int n_pad) {
        const int groups = n_pad / (kStates * (32 / kL));
        end = reinterpret_cast<float4*>(raw);
        fall = end + 2 * kMaxWarps * 32;
        a2 = fall + 2 * kMaxWarps * 32;
        h = a2 + groups * 32;
        b = reinterpret_cast<float*>(h + 2 * groups * 32);
        c = b + n_pad * (tile + 4);
        u = reinterpret_cast<T*>(c + n_pad * (tile + 4));
        dt = u + 2 * tile * kL;
        z = dt + 2 * tile * kL;
        rb = z + 2 * tile * kL;
        rc = rb + 2 * tile * n_pad;
    }
};

// kSplit: the blocks of a cluster take `per` tokens each of the same channels, twice: from zero (block 0: from
// h0) for the state at the end of their part, which the blocks after them read, and again from the state folded so.
template <typename T, int kL, bool kSplit>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) ttt_ssm_segments_kernel(const Params p, const int cblocks, const int n_pad, const int per) {
    constexpr int kQ = 32 / kL;
    constexpr int kOwn = kSeg / kQ;  // tokens whose elementwise work a lane does
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    const int rank = kSplit ? (int)cg::this_cluster().block_rank() : 0, ranks = kSplit ? (int)cg::this_cluster().num_blocks() : 1;
    const int block = (int)blockIdx.x / ranks, b = block / cblocks, c0 = block % cblocks * kL;
    const int ch = lane / kQ, part = lane % kQ, c = c0 + ch;
    const bool on = c < p.C;
    const int first_t = kSplit ? (int)min((long long)rank * per, (long long)p.T) : 0;
    const int T_own = kSplit ? min(p.T - first_t, per) : p.T;
    const int len = max(min(length_of(p.lengths, b, p.T) - first_t, T_own), 0);
    const long long row0 = (long long)b * p.T + first_t;
    const int tile = kSeg * warps, groups = n_pad / (kStates * kQ), pitch = tile + 4, shift = 31 - __clz(n_pad);
    const SegSmem<T, kL> s(smem_raw, tile, n_pad);
    const T* u_rows = static_cast<const T*>(p.u) + row0 * p.ld_u + c0;
    const T* dt_rows = static_cast<const T*>(p.dt) + row0 * p.ld_dt + c0;
    const T* z_rows = static_cast<const T*>(p.z) + row0 * p.ld_z + c0;
    const T* b_rows = static_cast<const T*>(p.Bm) + row0 * p.ld_b;
    const T* c_rows = static_cast<const T*>(p.Cm) + row0 * p.ld_c;
    T* y_rows = static_cast<T*>(p.y) + row0 * p.C + c;

    const auto stage = [&](int t0, int buf) {
        const int width = p.C - c0;
        stage_rows<T>(p.vec_rows, s.u + buf * tile * kL, u_rows, p.ld_u, t0, tile, len, kL, width, tid, threads);
        stage_rows<T>(p.vec_rows, s.dt + buf * tile * kL, dt_rows, p.ld_dt, t0, tile, len, kL, width, tid, threads);
        if (p.z) stage_rows<T>(p.vec_rows, s.z + buf * tile * kL, z_rows, p.ld_z, t0, tile, len, kL, width, tid, threads);
        stage_rows<T>(p.vec_bc, s.rb + buf * tile * n_pad, b_rows, p.ld_b, t0, tile, len, n_pad, p.N, tid, threads);
        stage_rows<T>(p.vec_bc, s.rc + buf * tile * n_pad, c_rows, p.ld_c, t0, tile, len, n_pad, p.N, tid, threads);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    for (int g = warp; g < groups; g += warps) {
        float h[kStates], v[kStates];
#pragma unroll
        for (int i = 0; i < kStates; i++) {
            const int n = (g * kQ + part) * kStates + i;
            h[i] = on && n < p.N && p.h0 && rank == 0 ? p.h0[((size_t)b * p.C + c) * p.N + n] : 0.f;
            v[i] = on && n < p.N ? rate(p.A[(size_t)c * p.N + n]) : 0.f;
        }
        s.h[g * 32 + lane] = make_float4(h[0], h[1], h[2], h[3]);
        s.a2[g * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
    }
    const float bias = on && p.dt_bias ? p.dt_bias[c] : 0.f, skip = on && p.D ? p.D[c] : 0.f;

    int turn = 0, buf = 0;  // turn: which of the two segment buffers
    float all_dt = 0.f;     // of the warp's tokens of all tiles
#pragma unroll 1
    for (int pass = kSplit ? 0 : 1; pass < 2; pass++) {
        const bool ends = kSplit && pass == 0;
        if (len > 0) stage(0, buf);
        for (int t0 = 0; t0 < len; t0 += tile, buf ^= 1) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
            if (t0 + tile < len) stage(t0 + tile, buf ^ 1);
            for (int i = tid; i < tile * n_pad; i += threads) {
                const int at = (i & (n_pad - 1)) * pitch + (i >> shift);
                s.b[at] = to_f32(s.rb[buf * tile * n_pad + i]);
                s.c[at] = to_f32(s.rc[buf * tile * n_pad + i]);
            }
            const int k0 = warp * kSeg;
            f2 dt2[kSeg / 2], du2[kSeg / 2], y2[kSeg / 2];  // of the warp's tokens, in pairs
            float own_u[kOwn], sum_dt = 0.f;
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
                float dt[kSeg], du[kSeg];
#pragma unroll
                for (int k = 0; k < kSeg; k++) {
                    if constexpr (kQ == 1) {
                        dt[k] = own_dt[k];
                        du[k] = own_dt[k] * own_u[k];
                    } else {
                        const int from = (lane & ~(kQ - 1)) + k / kOwn;
                        dt[k] = __shfl_sync(0xffffffffu, own_dt[k % kOwn], from);
                        du[k] = __shfl_sync(0xffffffffu, own_dt[k % kOwn] * own_u[k % kOwn], from);
                    }
                    sum_dt += dt[k];
                }
                all_dt += sum_dt;
#pragma unroll
                for (int k = 0; k < kSeg / 2; k++) {
                    dt2[k] = pack2(dt[2 * k], dt[2 * k + 1]);
                    du2[k] = pack2(du[2 * k], du[2 * k + 1]);
                    y2[k] = pack2(0.f, 0.f);
                }
            }
            __syncthreads();
            for (int g = 0; g < groups; g++, turn ^= 1) {
                const int n0 = (g * kQ + part) * kStates;
                const float4 A4 = s.a2[g * 32 + lane];
                const float a2[kStates] = {A4.x, A4.y, A4.z, A4.w};
                float a[kStates][kSeg], h[kStates];
                f2 in[kStates][kSeg / 2];
#pragma unroll
                for (int i = 0; i < kStates; i++) {
                    const f2 A2 = pack2(a2[i], a2[i]);
                    f2 x[kSeg / 2];
#pragma unroll
                    for (int k = 0; k < kSeg / 2; k++) x[k] = mul2(dt2[k], A2);
                    decays<true>(a[i], x);
                    const ulonglong2* Bi = reinterpret_cast<const ulonglong2*>(&s.b[(n0 + i) * pitch + k0]);
#pragma unroll
                    for (int k = 0; k < kSeg / 4; k++) {
                        const ulonglong2 Bk = Bi[k];
                        in[i][2 * k] = mul2(du2[2 * k], Bk.x);
                        in[i][2 * k + 1] = mul2(du2[2 * k + 1], Bk.y);
                    }
                    h[i] = 0.f;
#pragma unroll
                    for (int k = 0; k < kSeg / 2; k++) {
                        float lo, hi;
                        unpack2(in[i][k], lo, hi);
                        h[i] = fmaf(a[i][2 * k], h[i], lo);
                        h[i] = fmaf(a[i][2 * k + 1], h[i], hi);
                    }
                }
                s.end[(turn * kMaxWarps + warp) * 32 + lane] = make_float4(h[0], h[1], h[2], h[3]);
                // Decays of states that grow are left as their roots, as carried() takes them; for the others, where its product
                // and comparison a state and segment cost 6 %, as they are.
                const bool grows = warp_grows(p.softplus, a2);  // the same for all warps
                const float fall_dt = grows ? 0.5f * sum_dt : sum_dt;
                s.fall[(turn * kMaxWarps + warp) * 32 + lane] =
                    make_float4(decay(fall_dt * a2[0]), decay(fall_dt * a2[1]), decay(fall_dt * a2[2]), decay(fall_dt * a2[3]));
                __syncthreads();
                const float4 first = s.h[(buf * groups + g) * 32 + lane];
                h[0] = first.x;
                h[1] = first.y;
                h[2] = first.z;
                h[3] = first.w;
                const auto fold = [&](auto grow) {
                    for (int v = 0; v < warp + (ends ? 1 : 0); v++) {
                        const float4 e = s.end[(turn * kMaxWarps + v) * 32 + lane], f = s.fall[(turn * kMaxWarps + v) * 32 + lane];
                        const float es[kStates] = {e.x, e.y, e.z, e.w}, fs[kStates] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int i = 0; i < kStates; i++) h[i] = decltype(grow)::value ? carried(h[i], fs[i], fs[i], es[i]) : fmaf(fs[i], h[i], es[i]);
                    }
                };
                grows ? fold(std::true_type{}) : fold(std::false_type{});
                if (ends) {
                    if (warp == warps - 1) s.h[((buf ^ 1) * groups + g) * 32 + lane] = make_float4(h[0], h[1], h[2], h[3]);
                    continue;
                }
#pragma unroll
                for (int k = 0; k < kSeg / 4; k++) {
                    float hk[kStates][4];
#pragma unroll
                    for (int i = 0; i < kStates; i++) {
#pragma unroll
                        for (int q = 0; q < 2; q++) {
                            float lo, hi;
                            unpack2(in[i][2 * k + q], lo, hi);
                            hk[i][2 * q] = h[i] = fmaf(a[i][4 * k + 2 * q], h[i], lo);
                            hk[i][2 * q + 1] = h[i] = fmaf(a[i][4 * k + 2 * q + 1], h[i], hi);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kStates; i++) {
                        const ulonglong2 Ck = *reinterpret_cast<const ulonglong2*>(&s.c[(n0 + i) * pitch + k0 + 4 * k]);
                        y2[2 * k] = fma2(Ck.x, pack2(hk[i][0], hk[i][1]), y2[2 * k]);
                        y2[2 * k + 1] = fma2(Ck.y, pack2(hk[i][2], hk[i][3]), y2[2 * k + 1]);
                    }
                }
                if (warp == warps - 1) s.h[((buf ^ 1) * groups + g) * 32 + lane] = make_float4(h[0], h[1], h[2], h[3]);
            }
            if (ends) continue;
            float y[kSeg];
#pragma unroll
            for (int k = 0; k < kSeg / 2; k++) unpack2(y2[k], y[2 * k], y[2 * k + 1]);
            // a channel's lanes share out the tokens: kOwn sums each
            float own_y[kOwn];
            if constexpr (kQ == 1) {
#pragma unroll
                for (int j = 0; j < kOwn; j++) own_y[j] = y[j];
            } else {
                static_assert(kQ == 1 || kQ == 4, "two exchange steps");
                const bool up2 = part & 2, up1 = part & 1;
                float half[kSeg / 2];
#pragma unroll
                for (int j = 0; j < kSeg / 2; j++) {
                    const float keep = up2 ? y[kSeg / 2 + j] : y[j], send = up2 ? y[j] : y[kSeg / 2 + j];
                    half[j] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
                }
#pragma unroll
                for (int j = 0; j < kSeg / 4; j++) {
                    const float keep = up1 ? half[kSeg / 4 + j] : half[j], send = up1 ? half[j] : half[kSeg / 4 + j];
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
        if constexpr (kSplit) {
            if (!ends) continue;
            // the segments' buffers are free: the part's end states go to `end`, its decays to `fall`
            float* sums = reinterpret_cast<float*>(s.end);
            sums[warp * 32 + lane] = all_dt;
            __syncthreads();
            float total = 0.f;
            for (int v = 0; v < warps; v++) total += sums[v * 32 + lane];
            total *= 0.5f;
            __syncthreads();
            for (int g = warp; g < groups; g += warps) {
                const float4 A4 = s.a2[g * 32 + lane];
                s.end[g * 32 + lane] = s.h[(buf * groups + g) * 32 + lane];
                s.fall[g * 32 + lane] = make_float4(decay(total * A4.x), decay(total * A4.y), decay(total * A4.z), decay(total * A4.w));
            }
            cg::cluster_group cluster = cg::this_cluster();
            cluster.sync();
            for (int g = warp; g < groups && rank > 0; g += warps) {
                float4 h = cluster.map_shared_rank(s.end, 0)[g * 32 + lane];
                for (int r = 1; r < rank; r++) {
                    const float4 e = cluster.map_shared_rank(s.end, r)[g * 32 + lane], f = cluster.map_shared_rank(s.fall, r)[g * 32 + lane];
                    h = make_float4(carried(h.x, f.x, f.x, e.x), carried(h.y, f.y, f.y, e.y), carried(h.z, f.z, f.z, e.z), carried(h.w, f.w, f.w, e.w));
                }
                s.h[(buf * groups + g) * 32 + lane] = h;
            }
            if (rank == 0)
                for (int g = warp; g < groups; g += warps) {
                    float h[kStates];
#pragma unroll
                    for (int i = 0; i < kStates; i++) {
                        const int n = (g * kQ + part) * kStates + i;
                        h[i] = on && n < p.N && p.h0 ? p.h0[((size_t)b * p.C + c) * p.N + n] : 0.f;
                    }
                    s.h[(buf * groups + g) * 32 + lane] = make_float4(h[0], h[1], h[2], h[3]);
                }
            cluster.sync();  // the others have read this block's ends; and h0, which h_T may replace, has been read
        }
    }
    for (int g = warp; g < groups && rank == ranks - 1; g += warps) {  // the last block has the final state
        const float4 v = s.h[(buf * groups + g) * 32 + lane];
        const float h[kStates] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < kStates; i++) {
            const int n = (g * kQ + part) * kStates + i;
            if (on && n < p.N) p.h_T[((size_t)b * p.C + c) * p.N + n] = h[i];
        }
    }
    const float zero[1] = {0.f};
    for (int t = len + warp * kQ + part; t < T_own; t += warps * kQ)
        if (on) store_vec<1>(y_rows + (long long)t * p.C, zero);
}

template <typename T, int kL, bool kSplit>
cudaError_t start(const Params& p, int cblocks, int n_pad, int per, int ranks, int warps, size_t smem, cudaStream_t stream) {
    const auto kernel = ttt_ssm_segments_kernel<T, kL, kSplit>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.B * cblocks * ranks));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)ranks, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = kSplit ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p, cblocks, n_pad, per);
}

template <typename T, int kL>
cudaError_t launch(const SsmArgs& a, cudaStream_t stream) {
    const Params p = params_of(a);
    constexpr int step = kStates * (32 / kL);
    int n_pad = step;
    while (n_pad < a.N) n_pad *= 2;
    const long long cblocks = (a.C + kL - 1) / kL, grid = a.B * cblocks;
    if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
    // a warp for every 16 tokens, up to 8, and fewer where many states make the tile too large
    const int segs = (a.T + kSeg - 1) / kSeg;
    int warps = segs < 1 ? 1 : (segs < kMaxWarps ? segs : kMaxWarps);
    while (warps > 1 && SegSmem<T, kL>::bytes(kSeg * warps, n_pad) > kMaxSmem) warps--;
    const size_t smem = SegSmem<T, kL>::bytes(kSeg * warps, n_pad);
    const int tiles = (int)(((long long)a.T + kSeg * warps - 1) / (kSeg * warps));
    int ranks = 1;
    // Blocks of a cluster share out the tokens as long as all clusters run at once: 15 of eight blocks, 32 of four
    // (16 of eight, measured, take two turns).  A split walk reads its inputs twice, so two blocks gain a tenth (4096 tokens,
    // 512 channels, 16 states: 117 us against 131), four half (256: 63 against 131), eight three quarters (64: 35 against 131).
    while (ranks < 8 && 2 * ranks <= tiles && 2 * ranks * grid <= (ranks == 1 ? 148 : ranks == 2 ? 128 : 120)) ranks *= 2;
    if (ranks == 1) return start<T, kL, false>(p, (int)cblocks, n_pad, 0, 1, warps, smem, stream);
    return start<T, kL, true>(p, (int)cblocks, n_pad, (tiles + ranks - 1) / ranks * kSeg * warps, ranks, warps, smem, stream);
}

}  // namespace

cudaError_t launch_ssm_segments(const SsmArgs& a, int channels, cudaStream_t stream) {
    if (channels == 8) return a.dtype == TTT_BF16 ? launch<__nv_bfloat16, 8>(a, stream) : launch<float, 8>(a, stream);
    return a.dtype == TTT_BF16 ? launch<__nv_bfloat16, 32>(a, stream) : launch<float, 32>(a, stream);
}

}  // namespace ttt
