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
// bytes; the sum of squares and the largest |h w| (r > 0 scales it to the largest |y|) meet in one
// reduction, so 8 bits cost no second one.  Sums are in fp32; y, h, dh are rounded once.
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

struct NormParams {
    long long rows;
    int d;
    float eps;
    const void *x, *residual;
    const float* weight;
    void *y, *h;
    float* scale;  // 8 bits only
};

// V: elements a vector (16 bytes, or 1 where rows are not 16-byte aligned); kNV vectors a thread
template <typename T, int V, int kNV, bool kQ8>
__global__ void __launch_bounds__(1024) ttt_rmsnorm_kernel(const NormParams p) {
    __shared__ float2 s[32];
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;  // whole warps only: blockDim.y > 1 means one warp a row
    const size_t base = (size_t)row * p.d;
    const T* x = static_cast<const T*>(p.x) + base;
    const T* res = static_cast<const T*>(p.residual) + base;
    float h[kNV][V], g[kNV][V];
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int j = (threadIdx.x + i * blockDim.x) * V;
        if (j < p.d) {
            load_vec<V>(x + j, h[i]);
            if (p.residual) {
                float r[V];
                load_vec<V>(res + j, r);
#pragma unroll
                for (int k = 0; k < V; k++) h[i][k] += r[k];
            }
            load_vec<V>(p.weight + j, g[i]);
        } else {
#pragma unroll
            for (int k = 0; k < V; k++) h[i][k] = g[i][k] = 0.f;
        }
    }
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kNV; i++) {
#pragma unroll
        for (int k = 0; k < V; k++) {
            acc.x += h[i][k] * h[i][k];
            g[i][k] *= h[i][k];
            if (kQ8) acc.y = fmaxf(acc.y, fabsf(g[i][k]));
        }
    }
    acc = reduce_row<true>(acc, s);
    const float r = rsqrtf(acc.x / (float)p.d + p.eps);
    float inv = 1.f;  // y / scale = (h w) inv
    if (kQ8) {
        float scale = acc.y * r / kE4m3Max;
        inv = kE4m3Max / acc.y;  // r is in both
        if (r != r) {
            scale = inv = r;
        } else if (!(scale >= kScaleMin)) {
            scale = kScaleMin;
            inv = fminf(r * (1.f / kScaleMin), 3e38f);
        }
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int j = (threadIdx.x + i * blockDim.x) * V;
        if (j < p.d) {
            if (p.h) store_vec<V>(static_cast<T*>(p.h) + base + j, h[i]);
            float y[V];
#pragma unroll
            for (int k = 0; k < V; k++) y[k] = g[i][k] * (kQ8 ? inv : r);
            if constexpr (!kQ8) {
                store_vec<V>(static_cast<T*>(p.y) + base + j, y);
            } else {
                unsigned char* q = static_cast<unsigned char*>(p.y) + base + j;
                if constexpr (V == 8)
                    *reinterpret_cast<uint2*>(q) = make_uint2(pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7]));
                else if constexpr (V == 4)
                    *reinterpret_cast<uint32_t*>(q) = pack_e4m3(y[0], y[1], y[2], y[3]);
                else
                    *q = __nv_cvt_float_to_fp8(y[0], __NV_SATFINITE, __NV_E4M3);
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

// Groups walk the rows with a stride, so that a column's sum stays in registers until the end.
template <typename T, int V, int kNV>
__global__ void __launch_bounds__(1024) ttt_rmsnorm_backward_kernel(const NormBwdParams p) {
    __shared__ float2 s[2][32];
    const long long group = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const long long groups = (long long)gridDim.x * blockDim.y;
    float w[kNV][V], dw[kNV][V];
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int j = (threadIdx.x + i * blockDim.x) * V;
#pragma unroll
        for (int k = 0; k < V; k++) w[i][k] = dw[i][k] = 0.f;
        if (j < p.d) load_vec<V>(p.weight + j, w[i]);
    }
    int buf = 0;
    for (long long row = group; row < p.rows; row += groups, buf ^= 1) {
        const size_t base = (size_t)row * p.d;
        float h[kNV][V], dy[kNV][V], g[kNV][V];
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int j = (threadIdx.x + i * blockDim.x) * V;
#pragma unroll
            for (int k = 0; k < V; k++) h[i][k] = dy[i][k] = g[i][k] = 0.f;
            if (j < p.d) {
                load_vec<V>(static_cast<const T*>(p.h) + base + j, h[i]);
                load_vec<V>(static_cast<const T*>(p.dy) + base + j, dy[i]);
                if (p.dh_in) load_vec<V>(static_cast<const T*>(p.dh_in) + base + j, g[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kNV; i++)
#pragma unroll
            for (int k = 0; k < V; k++) {
                acc.x += h[i][k] * h[i][k];
                acc.y += dy[i][k] * w[i][k] * h[i][k];
            }
        acc = reduce_row<false>(acc, s[buf]);
        const float r = rsqrtf(acc.x / (float)p.d + p.eps);
        const float c = r * r * (acc.y / (float)p.d);
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int j = (threadIdx.x + i * blockDim.x) * V;
            if (j < p.d) {
                float o[V];
#pragma unroll
                for (int k = 0; k < V; k++) {
                    o[k] = r * (dy[i][k] * w[i][k] - h[i][k] * c) + g[i][k];
                    dw[i][k] += dy[i][k] * (h[i][k] * r);
                }
                store_vec<V>(static_cast<T*>(p.dh) + base + j, o);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int j = (threadIdx.x + i * blockDim.x) * V;
        if (j < p.d) store_vec<V>(p.partial + (size_t)group * p.d + j, dw[i]);
    }
}

struct Shape {
    int threads_x, threads_y, nv;
    bool vec;
};

// Threads a row: the fewest that hold it in one vector each, from a warp up; beyond 1024 threads kNV
// grows.  One warp a row packs four rows to a block.
Shape shape_of(int d, int es) {
    const int vec = 16 / es;
    Shape s{32, 4, 1, d % vec == 0};
    const int vecs = s.vec ? d / vec : d;
    if (vecs <= 32) return s;
    s.threads_y = 1;
    s.threads_x = 64;
    while (s.threads_x < 1024 && s.threads_x < vecs) s.threads_x *= 2;
    while (s.threads_x * s.nv < vecs) s.nv *= 2;
    return s;
}

template <typename F>
cudaError_t by_vectors(int nv, F f) {
    switch (nv) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        case 16: return f(std::integral_constant<int, 16>{});
        default: return cudaErrorInvalidValue;
    }
}

template <typename T, bool kQ8>
cudaError_t launch_forward(const NormParams& p, cudaStream_t stream) {
    const Shape s = shape_of(p.d, sizeof(T));
    const dim3 block(s.threads_x, s.threads_y);
    const long long blocks = (p.rows + s.threads_y - 1) / s.threads_y;
    return by_vectors(s.nv, [&](auto nv) {
        constexpr int kNV = decltype(nv)::value;
        constexpr int kV = Elem<T>::kVec;
        if (s.vec) {
            if constexpr (kNV <= 4) ttt_rmsnorm_kernel<T, kV, kNV, kQ8><<<(unsigned)blocks, block, 0, stream>>>(p);
        } else {
            ttt_rmsnorm_kernel<T, 1, kNV, kQ8><<<(unsigned)blocks, block, 0, stream>>>(p);
        }
        return cudaPeekAtLastError();
    });
}

// Column sums of `partial` [rows][cols]: 32 columns a block, 8 threads a column.  The order of the
// additions goes by the shape alone.
__global__ void __launch_bounds__(256) ttt_column_sum_kernel(int rows, int cols, const float* __restrict__ partial,
                                                             float* __restrict__ out) {
    __shared__ float s[8][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < cols)
        for (int r = threadIdx.y; r < rows; r += 8) a += partial[(size_t)r * cols + c];
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 8; i++) a += s[i][threadIdx.x];
        out[c] = a;
    }
}

// Row groups of the backward: enough blocks to fill 148 SMs with 1024 threads each, no more than rows.
long long backward_groups(long long rows, const Shape& s) {
    const long long per_block = s.threads_y;
    long long blocks = 148LL * (1024 / (s.threads_x * s.threads_y));
    const long long most = (rows + per_block - 1) / per_block;
    if (blocks > most) blocks = most;
    return blocks * per_block;
}

template <typename T>
cudaError_t launch_backward(const NormBwdParams& p, float* dweight, cudaStream_t stream) {
    const Shape s = shape_of(p.d, sizeof(T));
    const dim3 block(s.threads_x, s.threads_y);
    const long long groups = backward_groups(p.rows, s);
    cudaError_t e = by_vectors(s.nv, [&](auto nv) {
        constexpr int kNV = decltype(nv)::value;
        constexpr int kV = Elem<T>::kVec;
        const unsigned blocks = (unsigned)(groups / s.threads_y);
        if (s.vec) {
            if constexpr (kNV <= 4) ttt_rmsnorm_backward_kernel<T, kV, kNV><<<blocks, block, 0, stream>>>(p);
        } else {
            ttt_rmsnorm_backward_kernel<T, 1, kNV><<<blocks, block, 0, stream>>>(p);
        }
        return cudaPeekAtLastError();
    });
    if (e != cudaSuccess) return e;
    return launch_column_sum((int)groups, p.d, p.partial, dweight, stream);
}

}  // namespace

cudaError_t launch_column_sum(int rows, int cols, const float* partial, float* out, cudaStream_t stream) {
    ttt_column_sum_kernel<<<(cols + 31) / 32, dim3(32, 8), 0, stream>>>(rows, cols, partial, out);
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
    const Shape s = shape_of(d, dtype == TTT_BF16 ? 2 : 4);
    return (size_t)backward_groups((long long)B * T, s) * d * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, float* workspace, cudaStream_t stream) {
    const NormBwdParams p{(long long)a.B * a.T, a.d, a.eps, a.h, a.dy, a.dh_in, a.weight, a.dh, workspace};
    return a.dtype == TTT_BF16 ? launch_backward<__nv_bfloat16>(p, a.dweight, stream)
                               : launch_backward<float>(p, a.dweight, stream);
}

}  // namespace ttt
