// Root-mean-square norm over the residual stream, forward (with the residual's addition and an output
// in the input's type or in 8 bits) and backward.
//
//   h = x + residual,  r = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j r w_j
//   8 bits: scale = max(max_j |y_j| / 448, 2^-100),  q_j = e4m3(y_j / scale)
//   backward, with v_j = dy_j w_j and g the gradient that reaches h past the norm:
//     dh_j = r (v_j - h_j r^2 mean_i(v_i h_i)) + g_j,    dw_j = sum over rows of dy_j h_j r
//
// Both are bound by HBM: every element is read once and written once, kept in registers between.  A row
// belongs to one group of threads (a warp, or a block of 64 to 1024), each holding kNV vectors of 16
// bytes; a group walks rows with a stride, the next row on its way while one is worked on, and keeps its
// part of the weight.  The sum of squares and the largest |h w| (y / scale is h w 448 / max |h w|, without r)
// meet in one reduction, so 8 bits cost no second one.  Sums are in fp32; y, h, dh are rounded once.
//
// Where d is no multiple of a vector, rows start inside one: a group counts its vectors from the 16-byte
// boundary before its row, and the two at the ends go element by element.  The stride is a multiple of 8
// rows, so that all rows of a group start at the same place in a vector.
#include <cuda_fp8.h>

#include "block_internal.h"
#include "vec_io.cuh"

namespace ttt {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 7.888609052210118e-31f;  // 2^-100: a row of zeros has zeros and this scale

// Two values reduced over the row's threads at once: (sum, sum) or (sum, max).
template <bool kMax>
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    return make_float2(a.x + b.x, kMax ? fmaxf(a.y, b.y) : a.y + b.y);
}

// blockDim.x threads a row; blockDim.y > 1 only with blockDim.x = 32.  `s` is free again after the
// next __syncthreads, which a caller that reduces once per row of a loop gets from the double buffer.
template <bool kMax>
__device__ __forceinline__ float2 reduce_row(float2 v, float2* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = join<kMax>(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int i = 1; i < warps; i++) v = join<kMax>(v, s[i]);
    return v;
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Where a thread's i-th vector lies in its row, `off` elements past a 16-byte boundary
template <int V>
__device__ __forceinline__ int place(int i, int off) {
    return (int)(threadIdx.x + i * blockDim.x) * V - off;
}

struct NormParams {
    long long rows;
    int d;
    float eps;
    const void *x, *residual;
    const float* weight;
    void *y, *h;
    float* scale;  // 8 bits only
};

// A thread with one vector has room in 64 registers, so a row may have 1024 of them; with more vectors 512
constexpr int most_threads(int nv) { return nv == 1 ? 1024 : 512; }

template <typename T, int kNV, bool kQ8>
__global__ void __launch_bounds__(most_threads(kNV)) ttt_rmsnorm_kernel(const NormParams p) {
    constexpr int V = Elem<T>::kVec;
    __shared__ float2 s[2][32];
    const long long group = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const long long groups = (long long)gridDim.x * blockDim.y;
    if (group >= p.rows) return;  // whole warps only: blockDim.y > 1 means one warp a row
    const int off = (int)((size_t)group * p.d % V);
    const T* const x = static_cast<const T*>(p.x);
    const T* const res = static_cast<const T*>(p.residual);
    Raw<T, V> nx[kNV], nr[kNV];
    float w[kNV][V];
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int at = place<V>(i, off);
        nx[i].load_within(x + (size_t)group * p.d, at, p.d);
        if (res) nr[i].load_within(res + (size_t)group * p.d, at, p.d);
#pragma unroll
        for (int k = 0; k < V; k++) w[i][k] = at + k >= 0 && at + k < p.d ? p.weight[at + k] : 0.f;
    }
    int buf = 0;
    for (long long row = group; row < p.rows; row += groups, buf ^= 1) {
        const size_t base = (size_t)row * p.d;
        float h[kNV][V];
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            nx[i].get(h[i]);
            if (res) {
                float r[V];
                nr[i].get(r);
#pragma unroll
                for (int k = 0; k < V; k++) h[i][k] += r[k];
            }
            if (row + groups < p.rows) {
                const int at = place<V>(i, off);
                nx[i].load_within(x + base + (size_t)groups * p.d, at, p.d);
                if (res) nr[i].load_within(res + base + (size_t)groups * p.d, at, p.d);
            }
#pragma unroll
            for (int k = 0; k < V; k++) {
                acc.x += h[i][k] * h[i][k];
                if (kQ8) acc.y = fmaxf(acc.y, fabsf(h[i][k] * w[i][k]));
            }
        }
        acc = reduce_row<true>(acc, s[buf]);
        const float r = rsqrtf(acc.x / (float)p.d + p.eps);
        float factor = r;  // y, or y / scale, is (h w) factor
        if (kQ8) {
            float scale = acc.y * r / kE4m3Max;
            factor = kE4m3Max / acc.y;
            if (r != r) {
                scale = factor = r;
            } else if (!(scale >= kScaleMin)) {
                scale = kScaleMin;
                factor = fminf(r * (1.f / kScaleMin), 3e38f);
            }
            if (threadIdx.x == 0) p.scale[row] = scale;
        }
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int at = place<V>(i, off);
            if (at + V <= 0 || at >= p.d) continue;
            if (p.h) store_within<V>(static_cast<T*>(p.h) + base, at, p.d, h[i]);
            float y[V];
#pragma unroll
            for (int k = 0; k < V; k++) y[k] = h[i][k] * w[i][k] * factor;
            if constexpr (!kQ8) {
                store_within<V>(static_cast<T*>(p.y) + base, at, p.d, y);
            } else {
                unsigned char* q = static_cast<unsigned char*>(p.y) + base;
                if (at >= 0 && at + V <= p.d) {
                    if constexpr (V == 8)
                        *reinterpret_cast<uint2*>(q + at) =
                            make_uint2(pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7]));
                    else
                        *reinterpret_cast<uint32_t*>(q + at) = pack_e4m3(y[0], y[1], y[2], y[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < V; k++)
                        if (at + k >= 0 && at + k < p.d) q[at + k] = __nv_cvt_float_to_fp8(y[k], __NV_SATFINITE, __NV_E4M3);
                }
            }
        }
    }
}

struct NormBwdParams {
    long long rows;
    int d;
    float eps;
    const void *h, *dy, *dh_in;
    const float* weight;
    void* dh;
    float* partial;  // [groups][d]: each group's sum over its rows of dy h r
};

template <typename T, int kNV>
__global__ void __launch_bounds__(512) ttt_rmsnorm_backward_kernel(const NormBwdParams p) {
    constexpr int V = Elem<T>::kVec;
    __shared__ float2 s[2][32];
    const long long group = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const long long groups = (long long)gridDim.x * blockDim.y;
    const int off = (int)((size_t)group * p.d % V);
    const T* const hp = static_cast<const T*>(p.h);
    const T* const gp = static_cast<const T*>(p.dy);
    const T* const ip = static_cast<const T*>(p.dh_in);
    Raw<T, V> nh[kNV], ng[kNV], ni[kNV];
    float w[kNV][V], dw[kNV][V];
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int at = place<V>(i, off);
        if (group < p.rows) {
            nh[i].load_within(hp + (size_t)group * p.d, at, p.d);
            ng[i].load_within(gp + (size_t)group * p.d, at, p.d);
            if (ip) ni[i].load_within(ip + (size_t)group * p.d, at, p.d);
        }
#pragma unroll
        for (int k = 0; k < V; k++) {
            dw[i][k] = 0.f;
            w[i][k] = at + k >= 0 && at + k < p.d ? p.weight[at + k] : 0.f;
        }
    }
    int buf = 0;
    for (long long row = group; row < p.rows; row += groups, buf ^= 1) {
        const size_t base = (size_t)row * p.d, next = base + (size_t)groups * p.d;
        const bool more = row + groups < p.rows;
        float h[kNV][V], dy[kNV][V];
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            nh[i].get(h[i]);
            ng[i].get(dy[i]);
            if (more) {
                const int at = place<V>(i, off);
                nh[i].load_within(hp + next, at, p.d);
                ng[i].load_within(gp + next, at, p.d);
            }
#pragma unroll
            for (int k = 0; k < V; k++) {
                acc.x += h[i][k] * h[i][k];
                acc.y += dy[i][k] * w[i][k] * h[i][k];
            }
        }
        acc = reduce_row<false>(acc, s[buf]);
        const float r = rsqrtf(acc.x / (float)p.d + p.eps);
        const float c = r * r * (acc.y / (float)p.d);
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int at = place<V>(i, off);
            if (at + V <= 0 || at >= p.d) continue;
            float o[V], g[V];
            if (ip) {
                ni[i].get(g);
                if (more) ni[i].load_within(ip + next, at, p.d);
            }
#pragma unroll
            for (int k = 0; k < V; k++) {
                o[k] = r * (dy[i][k] * w[i][k] - h[i][k] * c) + (ip ? g[k] : 0.f);
                dw[i][k] += dy[i][k] * (h[i][k] * r);
            }
            store_within<V>(static_cast<T*>(p.dh) + base, at, p.d, o);
        }
    }
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int at = place<V>(i, off);
#pragma unroll
        for (int k = 0; k < V; k++)
            if (at + k >= 0 && at + k < p.d) p.partial[(size_t)group * p.d + at + k] = dw[i][k];
    }
}

struct Shape {
    int threads_x, threads_y, nv;
    long long blocks;
};

// Threads a row: the fewest that hold it in one vector each, from a warp up to `most`; past that 512 with
// more vectors.  One warp a row packs four rows to a block.  Blocks: `resident` threads on each of 148 SMs
// (1024 with 64 registers a thread, 768 with 80), or as many as there are rows; where rows start inside a
// vector, rounded down to a multiple of 8.
Shape shape_of(long long rows, int d, int es, int most, int resident) {
    const int v = 16 / es, vecs = d % v == 0 ? d / v : (d + 2 * v - 2) / v;
    Shape s{32, 4, 1, 0};
    if (vecs > 32) {
        s.threads_y = 1;
        s.nv = vecs <= most ? 1 : (vecs + 511) / 512;
        s.threads_x = ((vecs + s.nv - 1) / s.nv + 31) / 32 * 32;
    }
    const int a_block = s.threads_x * s.threads_y;
    s.blocks = 148LL * (a_block < resident ? resident / a_block : 1);
    if (d % v != 0) s.blocks -= s.blocks % 8;
    const long long need = (rows + s.threads_y - 1) / s.threads_y;
    if (s.blocks > need) s.blocks = need;  // one row a group at most
    return s;
}
Shape forward_shape(long long rows, int d, int es) { return shape_of(rows, d, es, 1024, 1024); }
Shape backward_shape(long long rows, int d, int es) { return shape_of(rows, d, es, 512, 768); }

template <typename F>
cudaError_t by_vectors(int nv, F f) {
    switch (nv) {
        case 1: f(std::integral_constant<int, 1>{}); break;
        case 2: f(std::integral_constant<int, 2>{}); break;
        case 3: f(std::integral_constant<int, 3>{}); break;
        case 4: f(std::integral_constant<int, 4>{}); break;
        case 5: f(std::integral_constant<int, 5>{}); break;
        case 6: f(std::integral_constant<int, 6>{}); break;
        case 7: f(std::integral_constant<int, 7>{}); break;
        case 8: f(std::integral_constant<int, 8>{}); break;
        case 9: f(std::integral_constant<int, 9>{}); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaPeekAtLastError();
}

template <typename T, bool kQ8>
cudaError_t launch_forward(const NormParams& p, cudaStream_t stream) {
    const Shape s = forward_shape(p.rows, p.d, sizeof(T));
    const dim3 block(s.threads_x, s.threads_y);
    return by_vectors(s.nv, [&](auto nv) {
        ttt_rmsnorm_kernel<T, decltype(nv)::value, kQ8><<<(unsigned)s.blocks, block, 0, stream>>>(p);
    });
}

// Column sums of `partial` [rows][cols]: 32 columns a block, 32 threads a column.  The order of the
// additions goes by the shape alone.
__global__ void __launch_bounds__(1024) ttt_column_sum_kernel(int rows, int cols, const float* __restrict__ partial,
                                                              float* __restrict__ out) {
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < cols)
        for (int r = threadIdx.y; r < rows; r += 32) a += partial[(size_t)r * cols + c];
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 32; i++) a += s[i][threadIdx.x];
        out[c] = a;
    }
}

template <typename T>
cudaError_t launch_backward(const NormBwdParams& p, float* dweight, cudaStream_t stream) {
    const Shape s = backward_shape(p.rows, p.d, sizeof(T));
    const dim3 block(s.threads_x, s.threads_y);
    cudaError_t e = by_vectors(s.nv, [&](auto nv) {
        ttt_rmsnorm_backward_kernel<T, decltype(nv)::value><<<(unsigned)s.blocks, block, 0, stream>>>(p);
    });
    if (e != cudaSuccess) return e;
    return launch_column_sum((int)(s.blocks * s.threads_y), p.d, p.partial, dweight, stream);
}

}  // namespace

cudaError_t launch_column_sum(int rows, int cols, const float* partial, float* out, cudaStream_t stream) {
    ttt_column_sum_kernel<<<(cols + 31) / 32, dim3(32, 32), 0, stream>>>(rows, cols, partial, out);
    return cudaPeekAtLastError();
}

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t stream) {
    const NormParams p{(long long)a.B * a.T, a.d, a.eps, a.x, a.residual, a.weight, a.y, a.h, a.scale};
    if (a.scale)
        return a.dtype == TTT_BF16 ? launch_forward<__nv_bfloat16, true>(p, stream) : launch_forward<float, true>(p, stream);
    return a.dtype == TTT_BF16 ? launch_forward<__nv_bfloat16, false>(p, stream) : launch_forward<float, false>(p, stream);
}

size_t rmsnorm_backward_workspace_bytes(int B, int T, int d, ttt_dtype dtype) {
    if (B < 1 || T < 1 || d < 1 || d > kNormMaxWidth) return 0;
    const Shape s = backward_shape((long long)B * T, d, dtype == TTT_BF16 ? 2 : 4);
    return (size_t)s.blocks * s.threads_y * d * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, float* workspace, cudaStream_t stream) {
    const NormBwdParams p{(long long)a.B * a.T, a.d, a.eps, a.h, a.dy, a.dh_in, a.weight, a.dh, workspace};
    return a.dtype == TTT_BF16 ? launch_backward<__nv_bfloat16>(p, a.dweight, stream)
                               : launch_backward<float>(p, a.dweight, stream);
}

}  // namespace ttt
