// Arguments and staging of the selective scan's kernels.
#pragma once

#include "block_internal.h"
#include "ssm_math.cuh"
#include "vec_io.cuh"

namespace ttt {
namespace ssm {

constexpr int kStates = 4;  // states a thread
constexpr size_t kMaxSmem = 227 * 1024;

struct Params {
    int B, T, C, N;
    long long ld_u, ld_dt, ld_b, ld_c, ld_z;
    int softplus;
    const void *u, *dt, *Bm, *Cm, *z;
    const float *dt_bias, *A, *D;
    const float* h0;
    const int* lengths;
    void* y;
    float* h_T;
    bool vec_rows, vec_bc;  // rows16 of u, dt and z, and of B and C
};

// Whether rows of `width` elements, `ld` apart, are whole 16-byte units on 16-byte boundaries
inline bool rows16(const void* q, long long ld, int width, int es) {
    return !q || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (ld * es) % 16 == 0 && (width * es) % 16 == 0);
}

inline Params params_of(const SsmArgs& a) {
    Params p{};
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
    const int es = a.dtype == TTT_BF16 ? 2 : 4;
    p.vec_rows = rows16(a.u, a.ld_u, a.C, es) && rows16(a.dt, a.ld_dt, a.C, es) && rows16(a.z, a.ld_z, a.C, es);
    p.vec_bc = rows16(a.Bm, a.ld_b, a.N, es) && rows16(a.Cm, a.ld_c, a.N, es);
    return p;
}

template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool live) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(live ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(live ? 4 : 0) : "memory");
}

template <typename T, bool kVec>
__device__ __forceinline__ void stage_rows_by(T* dst, const T* src, long long ld, int t0, int rows, int len, int cols, int width,
                                           int tid, int threads) {
    constexpr int kV = kVec ? 16 / (int)sizeof(T) : 1;
    const int per = max(cols / kV, 1), shift = 31 - __clz(per);  // pieces a row
    const auto put = [](T* to, const T* from, bool live) {
        if constexpr (kVec || sizeof(T) == 4)
            copy_async<kVec ? 16 : 4>(to, from, live);
        else
            *to = live ? *from : T(0.f);
    };
    if (per <= 32) {  // a thread keeps its column: `threads` is a multiple of 32
        const int c = (tid & (per - 1)) * kV, step = threads >> shift;
        int r = tid >> shift;
        const T* from = src + (long long)(t0 + r) * ld + c;
        T* to = dst + r * cols + c;
        const long long advance = step * ld;
        const int last = c < width ? len - t0 : 0;
        if constexpr (kVec || sizeof(T) == 4) {
            for (; r < rows; r += step, from += advance, to += step * cols) put(to, r < last ? from : src, r < last);
        } else {
            // there is no asynchronous copy of two bytes: eight loads on their way before the first is stored
            for (; r < rows; r += 8 * step, from += 8 * advance, to += 8 * step * cols) {
                T v[8];
#pragma unroll
                for (int k = 0; k < 8; k++) v[k] = r + k * step < last ? from[k * advance] : T(0.f);
#pragma unroll
                for (int k = 0; k < 8; k++)
                    if (r + k * step < rows) to[k * step * cols] = v[k];
            }
        }
    } else {
        for (int i = tid; i < rows * per; i += threads) {
            const int r = i >> shift, c = (i & (per - 1)) * kV;
            const bool live = t0 + r < len && c < width;
            put(dst + r * cols + c, live ? src + (long long)(t0 + r) * ld + c : src, live);
        }
    }
}

// Rows [t0, t0 + rows) of `cols` (a power of two) columns into shared memory (row stride `cols`); rows at or
// past `len` and columns at or past `width` become zeros and are not read.  vec: 16 bytes a copy (rows16 of
// the rows); else an element, which for bf16 cp.async cannot copy.
template <typename T>
__device__ __forceinline__ void stage_rows(bool vec, T* dst, const T* src, long long ld, int t0, int rows, int len, int cols,
                                           int width, int tid, int threads) {
    if (vec)
        stage_rows_by<T, true>(dst, src, ld, t0, rows, len, cols, width, tid, threads);
    else
        stage_rows_by<T, false>(dst, src, ld, t0, rows, len, cols, width, tid, threads);
}

}  // namespace ssm

// The scan with the states shared out among the warps (ttt_ssm_scan.cu; N <= 16) and with the tokens shared out
// (ttt_ssm_segments.cu; kL = 8 or 32 channels a block)
cudaError_t launch_ssm_scan(const SsmArgs& a, cudaStream_t stream);
cudaError_t launch_ssm_segments(const SsmArgs& a, int channels, cudaStream_t stream);

}  // namespace ttt
