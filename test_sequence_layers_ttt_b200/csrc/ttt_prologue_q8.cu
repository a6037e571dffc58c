// The TTT layer's prologue from 8-bit operands: Q, K, V and eta of ttt_prologue.cu from x and weights in
// e4m3, x with a scale a token (as the 8-bit norm writes it), the weights with a scale an output feature.
//
// One GEMM with the tokens as rows, [B*T, d_model] x [d_model, 3 H d + H], both operands K-major; the sum
// over d_model is of exact products in fp32, and the scales, constant along it, multiply the accumulator in
// the epilogue, before the rotary embedding (of Q and K) or the sigmoid gate.  Column tiles of 256 hold four
// heads of one of Q, K, V; one more tile of round16(H) columns holds the H learning-rate logits.  Persistent
// CTAs of 12 warps walk the tiles (column tiles fastest, so the CTAs in flight share each row tile in L2):
//   warp 0     TMA loads of x (128 x 128) and weight (256 x 128) tiles, 4-stage ring; past d_model a box
//              reads zeros
//   warp 1     TMEM allocation and the tcgen05 MMAs (kind f8f6f4, M = 128, N = 256, K = 32), fp32
//              accumulators in two TMEM buffers of 256 columns
//   warps 4-11 the epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31, one token row a thread, and two of the
//              tile's four heads; a head's rows go out by TMA from a swizzled stage in shared memory
// While the epilogue drains one accumulator the MMA warp fills the other.  Every wait is bounded: after
// about a second without progress the kernel records an error word and stops waiting (outputs undefined;
// TTT_ERR_TIMEOUT with TTT_CHECK=1).
//
// Measured (2 x 32768 tokens, d_model 2048, 32 heads): 0.69 to 0.72 ms, 2.4 PFLOP/s, and 0.81 to 0.83 ms in a long run
// of calls, when the power cap lowers the clock; without the epilogue's work 0.52 ms, with all of it but the stores
// 0.58 ms.  One token of 64 streams: 14.6 us, 25 tiles on as many SMs.  The tensor pipe is busy for 67 % of the clocks,
// and each CTA takes 48 KB of operands a K step through the L2, 10 GB in all.  Eight epilogue warps instead
// of four, TMA stores and angles in fixed point took it there from 1.04 ms; a tile of 256 tokens in one CTA gave nothing.
#include <cstdlib>

#include "block_internal.h"
#include "common.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"
#include "vec_io.cuh"

namespace ttt {

__device__ unsigned int g_prologue_q8_error_word = 0;

namespace {

constexpr int kD = 64;               // head dimension
constexpr int kBM = 128, kBK = 128;  // tile rows (tokens), K step per stage (bytes = elements)
constexpr int kBN = 256;             // four heads of 64
constexpr int kStages = 4;
constexpr int kEpilogue = 8;  // warps
constexpr int kThreads = 128 + 32 * kEpilogue;
constexpr uint32_t kTmemCols = 512;  // two accumulators of 256 columns
constexpr long long kTimeoutCycles = 2000000000LL;

struct alignas(1024) PStage {
    unsigned char A[kBM * kBK];  // x tile [128 tokens][128 k], 128-byte swizzle (K-major)
    unsigned char B[kBN * kBK];  // weights [256 features][128 k], or theta_lr [Hp][128 k]
};

struct ProSmem {
    PStage st[kStages];
    unsigned char out[kEpilogue][32 * kD * 2];  // a warp's rows of one head on their way out, 128-byte swizzle
    unsigned long long turn[kD / 2];  // base^(-2i/d) / (2 pi), in turns of 2^64
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
};

// Instruction descriptor of kind::f8f6f4: fp32 accumulator, A and B e4m3 (format 0), both K-major
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (int spins = 1;; spins++) {
        if (*abort_flag) return false;
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((spins & 63) == 0 && clock64() - t0 > kTimeoutCycles) {
            *abort_flag = 1;
            atomicOr(&g_prologue_q8_error_word, 1u);
            return false;
        }
    }
}

__device__ __forceinline__ void ld_32x32b_x16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}

// A box of shared memory (the generic proxy's writes of it fenced) to global memory; rows past the tensor's end
// are left out.  One thread; `read_out` waits until the shared memory may be written again, `all_out` for the
// stores themselves.
__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tmap),
                 "r"(ptx::smem_addr(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void read_out() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void all_out() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct PrologueQ8Params {
    int B, T, H, d_model, pos0, rotary, n_col_tiles, n_tiles, hp;  // hp: H rounded up to 16
    float eta_base, rope_base;
    const float *scale_x, *scale_q, *scale_k, *scale_v, *scale_lr, *b_lr;
    __nv_bfloat16 *Q, *K, *V;
    float* eta;
};

__global__ void __launch_bounds__(kThreads, 1)
ttt_prologue_q8_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmWq,
                       const __grid_constant__ CUtensorMap tmWk, const __grid_constant__ CUtensorMap tmWv,
                       const __grid_constant__ CUtensorMap tmWl, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const PrologueQ8Params p) {
    extern __shared__ unsigned char smem_raw[];
    ProSmem& s = *reinterpret_cast<ProSmem*>(smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort_flag = &s.abort_flag;
    const int nk = (p.d_model + kBK - 1) / kBK;  // the last step past d_model reads zeros
    const int M = p.B * p.T;
    const int groups = p.H / 4;  // column tiles per projection
    if (tid == 0) {
        s.abort_flag = 0;
        for (int i = 0; i < kStages; i++) {
            ptx::mbar_init(&s.full[i], 1);
            ptx::mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            ptx::mbar_init(&s.acc_full[i], 1);
            ptx::mbar_init(&s.acc_empty[i], kEpilogue);
        }
        ptx::mbar_init(&s.drain, 1);
        ptx::fence_mbar_init();
    }
    if (warp == 1) tc05::tmem_alloc(ptx::smem_addr(&s.tmem_base), kTmemCols);
    if (tid < kD / 2)  // the constant is 2^64 / (2 pi); 64 in the exponent would cost the double four bits
        s.turn[tid] = (unsigned long long)(exp2(-(2.0 * tid / kD) * log2((double)p.rope_base)) * 2935890503282001226.0);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = s.tmem_base;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            ptx::prefetch_tmap(&tmX);
            ptx::prefetch_tmap(&tmWq);
            ptx::prefetch_tmap(&tmWk);
            ptx::prefetch_tmap(&tmWv);
            ptx::prefetch_tmap(&tmWl);
            long long it = 0;
            int inflight = 0;
            for (int tile = blockIdx.x; tile < p.n_tiles && !*abort_flag; tile += gridDim.x) {
                const int mt = tile / p.n_col_tiles, ct = tile % p.n_col_tiles;
                const int proj = ct / groups, grp = ct % groups;  // proj 3: the learning-rate tile
                const void* tmW = proj == 0 ? &tmWq : proj == 1 ? &tmWk : proj == 2 ? &tmWv : &tmWl;
                const uint32_t bytes = kBM * kBK + (proj == 3 ? p.hp : kBN) * kBK;
                for (int kb = 0; kb < nk; kb++, it++) {
                    const int st = (int)(it % kStages);
                    if (it >= kStages && !wait_bounded(&s.empty[st], (uint32_t)(((it / kStages) - 1) & 1),
                                                       abort_flag))
                        break;
                    ptx::mbar_arrive_expect_tx(&s.full[st], bytes);
                    ptx::tma_load_2d(s.st[st].A, &tmX, &s.full[st], kb * kBK, mt * kBM);
                    ptx::tma_load_2d(s.st[st].B, tmW, &s.full[st], kb * kBK, proj == 3 ? 0 : grp * kBN);
                    inflight = it + 1 < kStages ? (int)(it + 1) : kStages;
                }
            }
            // drain own loads: the last `inflight` stages
            for (long long j = it - 1; j >= 0 && j >= it - inflight; j--) {
                const long long t0 = clock64();
                while (!ptx::mbar_try_wait(&s.full[j % kStages], (uint32_t)((j / kStages) & 1))) {
                    if (clock64() - t0 > 4 * kTimeoutCycles) {
                        atomicOr(&g_prologue_q8_error_word, 2u);
                        break;
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            const uint32_t i_qkv = idesc_e4m3(kBM, kBN);
            const uint32_t i_lr = idesc_e4m3(kBM, p.hp);
            long long it = 0;
            int local = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < p.n_tiles && ok; tile += gridDim.x, local++) {
                const int ct = tile % p.n_col_tiles;
                const bool lr = ct / groups == 3;
                const int buf = local & 1;
                if (local >= 2) ok = wait_bounded(&s.acc_empty[buf], (uint32_t)(((local >> 1) - 1) & 1), abort_flag);
                if (!ok) break;
                tc05::fence_after_sync();
                const uint32_t d = tmem + (uint32_t)(buf * kBN);
                for (int kb = 0; kb < nk; kb++, it++) {
                    const int st = (int)(it % kStages);
                    ok = wait_bounded(&s.full[st], (uint32_t)((it / kStages) & 1), abort_flag);
                    if (!ok) break;
                    tc05::fence_after_sync();
                    const uint32_t a = ptx::smem_addr(s.st[st].A), b = ptx::smem_addr(s.st[st].B);
#pragma unroll
                    for (int ks = 0; ks < kBK / 32; ks++)
                        mma_e4m3(d, tc05::desc_k128(a, ks), tc05::desc_k128(b, ks), lr ? i_lr : i_qkv,
                                 (kb > 0 || ks > 0) ? 1u : 0u);
                    tc05::commit(ptx::smem_addr(&s.empty[st]));
                }
                if (!ok) break;
                tc05::commit(ptx::smem_addr(&s.acc_full[buf]));
            }
            tc05::commit(ptx::smem_addr(&s.drain));
            const long long t0 = clock64();
            while (!ptx::mbar_try_wait(&s.drain, 0)) {
                if (clock64() - t0 > 4 * kTimeoutCycles) {
                    atomicOr(&g_prologue_q8_error_word, 4u);
                    break;
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue
        const int q = warp % 4, half = (warp - 4) / 4;  // TMEM lanes 32 q ..; heads 2 half and 2 half + 1
        const uint32_t tq = tmem + tc05::taddr_lane(32 * q);
        const float inv_d = 1.f / kD;
        int local = 0;
        for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x, local++) {
            const int mt = tile / p.n_col_tiles, ct = tile % p.n_col_tiles;
            const int proj = ct / groups, grp = ct % groups;
            const int buf = local & 1;
            wait_bounded(&s.acc_full[buf], (uint32_t)((local >> 1) & 1), abort_flag);
            tc05::fence_after_sync();
            const int m = mt * kBM + 32 * q + lane;  // this thread's token row
            const bool valid = m < M;
            const int bb = valid ? m / p.T : 0, t = valid ? m % p.T : 0;
            const uint32_t tacc = tq + (uint32_t)(buf * kBN);
            const float sx = valid ? p.scale_x[m] : 0.f;
            if (proj == 3) {
                // learning-rate logits: columns 0..H-1
                for (int c0 = 16 * half; c0 < p.hp; c0 += 32) {  // hp is a multiple of 16, at most 256
                    float v[16];
                    ld_32x32b_x16(tacc + (uint32_t)c0, v);
                    tc05::wait_ld();
                    for (int j = 0; j < 16 && c0 + j < p.H; j++) {
                        const int hh = c0 + j;
                        const float logit = v[j] * (sx * p.scale_lr[hh]) + p.b_lr[hh];
                        if (valid)
                            p.eta[((size_t)bb * p.H + hh) * p.T + t] = p.eta_base * inv_d / (1.f + __expf(-logit));
                    }
                }
            } else {
                __nv_bfloat16* out = proj == 0 ? p.Q : proj == 1 ? p.K : p.V;
                const float* sw = (proj == 0 ? p.scale_q : proj == 1 ? p.scale_k : p.scale_v) + grp * kBN;
                const bool rope = p.rotary && proj < 2;
                // the rotation of this token row, shared by the tile's four heads, times the token's scale: angle
                // pos * base^(-2i/d) in fixed point, whose overflow leaves whole turns out, then sin and cos by the
                // special-function unit: the angle is off by half of 2^-23 turns, 3.7e-7, and by the step's rounding,
                // pos 2^-54 turns (2e-11 at position 50000, 7e-7 near 2^31), and they by 5e-7 at most, against the
                // outputs' half step of 2^-8.  (In double the reduction took as long as both functions.)
                f2 cs[16], sn[16];  // of two neighbouring features each
                if (rope) {
                    const unsigned long long pos = (unsigned long long)((long long)p.pos0 + t);
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        float c[2], n[2];
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            // the fraction of a turn to the nearest 2^-23, a float in [-1/2, 1/2); what passes 1/2 comes
                            // back at -1/2, the same angle
                            const uint32_t phase = (uint32_t)((pos * s.turn[2 * i + k]) >> 32) + 0x80000100u;
                            const float r = (__uint_as_float(0x3f800000u | (phase >> 9)) - 1.5f) * 6.283185307179586f;
                            c[k] = sx * __cosf(r);
                            n[k] = sx * __sinf(r);
                        }
                        cs[i] = pack2(c[0], c[1]);
                        sn[i] = pack2(n[0], n[1]);
                    }
                }
                // The warp's rows are neighbours in Q, K, V unless a sequence ends among them: then one box
                // takes a head's rows out, and rows past the sequence's (and the batch's) end fall away.
                const int bb0 = __shfl_sync(0xffffffffu, bb, 0), t0 = __shfl_sync(0xffffffffu, t, 0);
                const bool one_box = __all_sync(0xffffffffu, !valid || bb == bb0) && mt * kBM + 32 * q < M;
                const void* tmO = proj == 0 ? &tmQ : proj == 1 ? &tmK : &tmV;
                unsigned char* stage = s.out[warp - 4];
                const f2 sx2 = pack2(sx, sx), minus = pack2(-1.f, -1.f);
                for (int hh4 = 2 * half; hh4 < 2 * half + 2; hh4++) {
                    const int head = 4 * grp + hh4;
                    uint4* dst = reinterpret_cast<uint4*>(out + (((size_t)bb * p.H + head) * p.T + t) * kD);
                    if (lane == 0) read_out();
                    __syncwarp();
#pragma unroll
                    for (int f = 0; f < 32; f += 16) {  // features f .. f + 15 and their partners 32 further
                        float x1[16], x2[16];
                        ld_32x32b_x16(tacc + (uint32_t)(64 * hh4 + f), x1);
                        ld_32x32b_x16(tacc + (uint32_t)(64 * hh4 + 32 + f), x2);
                        const ulonglong2* w4 = reinterpret_cast<const ulonglong2*>(sw + 64 * hh4 + f);
                        f2 wa[8], wb[8];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const ulonglong2 a = w4[i], b = w4[8 + i];
                            wa[2 * i] = a.x;
                            wa[2 * i + 1] = a.y;
                            wb[2 * i] = b.x;
                            wb[2 * i + 1] = b.y;
                        }
                        tc05::wait_ld();
                        uint32_t o1[8], o2[8];
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            const f2 u = mul2(pack2(x1[2 * k], x1[2 * k + 1]), wa[k]);
                            const f2 v = mul2(pack2(x2[2 * k], x2[2 * k + 1]), wb[k]);
                            f2 y1, y2;
                            if (rope) {
                                const f2 c = cs[f / 2 + k], n = sn[f / 2 + k];
                                y1 = fma2(mul2(v, minus), n, mul2(u, c));
                                y2 = fma2(u, n, mul2(v, c));
                            } else {
                                y1 = mul2(u, sx2);
                                y2 = mul2(v, sx2);
                            }
                            float lo, hi;
                            unpack2(y1, lo, hi);
                            o1[k] = pack_bf16(lo, hi);
                            unpack2(y2, lo, hi);
                            o2[k] = pack_bf16(lo, hi);
                        }
#pragma unroll
                        for (int c = 0; c < 2; c++) {  // 16-byte chunks f / 8 + c and 4 + f / 8 + c of the row
                            const uint4 a = make_uint4(o1[4 * c], o1[4 * c + 1], o1[4 * c + 2], o1[4 * c + 3]);
                            const uint4 b = make_uint4(o2[4 * c], o2[4 * c + 1], o2[4 * c + 2], o2[4 * c + 3]);
                            if (one_box) {
                                *reinterpret_cast<uint4*>(stage + lane * 128 + (((f / 8 + c) ^ (lane & 7)) * 16)) = a;
                                *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 + f / 8 + c) ^ (lane & 7)) * 16)) = b;
                            } else if (valid) {
                                dst[f / 8 + c] = a;
                                dst[4 + f / 8 + c] = b;
                            }
                        }
                    }
                    if (one_box) {
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store_3d(tmO, stage, 0, t0, bb0 * p.H + head);
                    }
                }
            }
            tc05::fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s.acc_empty[buf]);
        }
        if (lane == 0) all_out();
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    if (warp == 1) tc05::tmem_dealloc(tmem, kTmemCols);
}

// [rows][inner] e4m3 in boxes of [box_rows][128] with the 128-byte swizzle
bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {inner, rows};
    cuuint64_t strides[1] = {inner};
    cuuint32_t box[2] = {kBK, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [BH][T][64] bf16 in boxes of [1][32][64] with the 128-byte swizzle
bool make_out_map(CUtensorMap* m, void* base, int T, long long BH) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {kD, (cuuint64_t)T, (cuuint64_t)BH};
    cuuint64_t strides[2] = {kD * 2, (cuuint64_t)T * kD * 2};
    cuuint32_t box[3] = {kD, 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool prologue_q8_supports(int B, int T, int H, int d, int d_model) {
    return B >= 1 && T >= 1 && d == kD && d_model >= 16 && d_model % 16 == 0 && H >= 4 && H % 4 == 0 && H <= 256 &&
           (long long)B * T < (1LL << 31) - kBM &&
           ((long long)B * T + kBM - 1) / kBM * (3 * (H / 4) + 1) < (1LL << 31) - 1024;
}

cudaError_t launch_prologue_q8(const PrologueArgs& a, const PrologueScales& s, cudaStream_t stream) {
    if (!prologue_q8_supports(a.B, a.T, a.H, a.d, a.d_model)) return cudaErrorInvalidValue;
    const int M = a.B * a.T, hp = (a.H + 15) / 16 * 16;
    const uint64_t dm = (uint64_t)a.d_model, features = (uint64_t)a.H * kD;
    CUtensorMap mx, mq, mk, mv, ml;
    if (!make_map(&mx, a.x, dm, (uint64_t)M, kBM) || !make_map(&mq, a.theta_q, dm, features, kBN) ||
        !make_map(&mk, a.theta_k, dm, features, kBN) || !make_map(&mv, a.theta_v, dm, features, kBN) ||
        !make_map(&ml, a.theta_lr, dm, (uint64_t)a.H, (uint32_t)hp))
        return cudaErrorInvalidValue;
    CUtensorMap oq, ok, ov;
    const long long BH = (long long)a.B * a.H;
    if (!make_out_map(&oq, a.Q, a.T, BH) || !make_out_map(&ok, a.K, a.T, BH) || !make_out_map(&ov, a.V, a.T, BH))
        return cudaErrorInvalidValue;
    PrologueQ8Params p{};
    p.B = a.B;
    p.T = a.T;
    p.H = a.H;
    p.d_model = a.d_model;
    p.pos0 = a.pos0;
    p.rotary = a.rotary;
    p.n_col_tiles = 3 * (a.H / 4) + 1;
    p.n_tiles = (int)(((long long)M + kBM - 1) / kBM) * p.n_col_tiles;
    p.hp = hp;
    p.eta_base = a.eta_base;
    p.rope_base = a.rope_base;
    p.scale_x = s.x;
    p.scale_q = s.q;
    p.scale_k = s.k;
    p.scale_v = s.v;
    p.scale_lr = s.lr;
    p.b_lr = a.b_lr;
    p.Q = static_cast<__nv_bfloat16*>(a.Q);
    p.K = static_cast<__nv_bfloat16*>(a.K);
    p.V = static_cast<__nv_bfloat16*>(a.V);
    p.eta = a.eta;
    const size_t smem = sizeof(ProSmem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(ttt_prologue_q8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int grid = p.n_tiles < sms ? p.n_tiles : sms;
    ttt_prologue_q8_kernel<<<grid, kThreads, smem, stream>>>(mx, mq, mk, mv, ml, oq, ok, ov, p);
    return cudaPeekAtLastError();
}

cudaError_t read_and_clear_prologue_q8_error(unsigned int* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_prologue_q8_error_word, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_prologue_q8_error_word, &zero, sizeof(unsigned int));
}

}  // namespace ttt
