// Root-mean-square norm over the residual stream, forward (with the residual's addition and an output
// in the input's type or in 8 bits) and backward.
//
//   h = x + residual,  r = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j r w_j
//   8 bits: scale = max(max_j |y_j| / 448, 2^-100),  q_j = e4m3(y_j / scale)
//   backward, with v_j = dy_j w_j and g the gradient that reaches h past the norm:
//     dh_j = r (v_j - h_j r^2 mean_i(v_i h_i)) + g_j,    dw_j = sum over rows of dy_j h_j r
//
// Both are bound by HBM: every element is read once and written once, kept in registers between.  A row
// belongs to one group of threads (a part of a warp, a warp, or a block of up to 512), each holding kNV vectors of 16 bytes,
// 16 elements where the row is long enough: with 8 the reduction, some 70 instructions a thread and row, took
// as many as the elements.  A group walks rows with a stride and keeps its part of the weight; in the forward
// the next row is on its way while one is worked on, and so it is in the backward of 16-bit rows; that of fp32 rows,
// whose registers are full, has other blocks of the SM.  The sum of squares and the largest |h w| (y / scale is h w 448 / max |h w|,
// without r) meet in one reduction, so 8 bits cost no second one.  Sums are in fp32; y, h, dh are rounded once.
//
// Measured: 2 x 32768 rows of 2048, bf16 with a residual and an 8-bit output, 165 us, 5.7 TB/s, 0.87 of the copy
// bandwidth; gradient of 32768 rows of 2048 in bf16 95 us, 0.86 of it; of 3 x 2731 rows of 2047 in fp32, rows that start
// inside a vector, 68 us, 4.0 TB/s: three blocks an SM, all that its registers hold, leave the memory waiting in the
// reductions.  4096 rows of 9001 in fp32 97 us forward (0.92) and 164 backward (0.55, one block an SM).  Two blocks of 512
// threads an SM leave the 16-bit forward 64 registers a thread, and its main variant spills 32 to 56 bytes.
//
// Where d is no multiple of a vector (kShift), rows start inside one: a group counts its vectors from the
// 16-byte boundary before its row, and the two at the ends go element by element.  The stride is a multiple of
// 8 rows, so that all rows of a group start at the same place in a vector.
#include <cuda_fp8.h>

#include "block_internal.h"
#include "vec_io.cuh"

#include <type_traits>

namespace ttt {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 7.888609052210118e-31f;  // 2^-100: a row of zeros has zeros and this scale

// The larger one, NaN where either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two values reduced over the row's threads at once: (sum, sum) or (sum, max).
template <bool kMax>
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    return make_float2(a.x + b.x, kMax ? max_nan(a.y, b.y) : a.y + b.y);
}

// blockDim.x threads a row: a power of two up to a warp, or whole warps.  `s` is free again after the next
// __syncthreads, which a caller that reduces once per row of a loop gets from the double buffer.
template <bool kMax>
__device__ __forceinline__ float2 reduce_row(float2 v, float2* s) {
    for (int o = min((int)blockDim.x, 32) / 2; o > 0; o >>= 1)
        v = join<kMax>(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    const int warps = blockDim.x >> 5;
    if (warps <= 1) return v;
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
template <bool kShift, typename T, int V>
__device__ __forceinline__ void load_at(Raw<T, V>& r, const T* row, int at, int d) {
    if constexpr (kShift) {
        r.load_within(row, at, d);
    } else if (at < d) {
        r.load(row + at);
    } else {
#pragma unroll
        for (int i = 0; i < Raw<T, V>::kWords; i++) r.w[i] = 0u;
    }
}
template <bool kShift, int V, typename T>
__device__ __forceinline__ void store_at(T* row, int at, int d, const f2 (&o)[V / 2]) {
    float v[V];
    from_pairs<V>(o, v);
    if constexpr (kShift)
        store_within<V>(row, at, d, v);
    else
        store_vec<V>(row + at, v);
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

template <typename T, int kNV, bool kShift, bool kQ8>
__global__ void __launch_bounds__(512, sizeof(T) == 2 && kNV <= 2 ? 2 : 1) ttt_rmsnorm_kernel(const NormParams p) {
    constexpr int V = Elem<T>::kVec, P = V / 2;
    __shared__ float2 s[2][16];
    const long long group = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const long long groups = (long long)gridDim.x * blockDim.y;
    const int off = kShift ? (int)((size_t)group * p.d % V) : 0;
    const T* x = static_cast<const T*>(p.x) + (size_t)group * p.d;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + (size_t)group * p.d : nullptr;
    const size_t stride = (size_t)groups * p.d;
    Raw<T, V> nx[kNV], nr[kNV];
    f2 w[kNV][P];
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int at = place<V>(i, off), d = group < p.rows ? p.d : -V;
        load_at<kShift>(nx[i], x, at, d);
        if (res) load_at<kShift>(nr[i], res, at, d);
    }
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int at = place<V>(i, off);
        float v[V];
#pragma unroll
        for (int k = 0; k < V; k++) v[k] = at + k >= 0 && at + k < p.d ? p.weight[at + k] : 0.f;
        to_pairs<V>(v, w[i]);
    }
    int buf = 0;
    // all rows of a block go round together; one past the end has zeros and writes nothing
    for (long long row = group; row - threadIdx.y < p.rows; row += groups, buf ^= 1) {
        const size_t base = (size_t)row * p.d;
        const int d = row < p.rows ? p.d : -V;
        f2 h[kNV][P], sq = pack2(0.f, 0.f);
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            pairs_of(nx[i], h[i]);
            if (res) {
                f2 r[P];
                pairs_of(nr[i], r);
#pragma unroll
                for (int k = 0; k < P; k++) h[i][k] = add2(h[i][k], r[k]);
            }
        }
        x += stride;
        if (res) res += stride;
        if (row - threadIdx.y + groups < p.rows) {
            const int next = row + groups < p.rows ? p.d : -V;
#pragma unroll
            for (int i = 0; i < kNV; i++) {
                const int at = place<V>(i, off);
                load_at<kShift>(nx[i], x, at, next);
                if (res) load_at<kShift>(nr[i], res, at, next);
            }
        }
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int at = place<V>(i, off);
            if (p.h && at < d && at + V > 0) store_at<kShift, V>(static_cast<T*>(p.h) + base, at, d, h[i]);
#pragma unroll
            for (int k = 0; k < P; k++) {
                sq = fma2(h[i][k], h[i][k], sq);
                h[i][k] = mul2(h[i][k], w[i][k]);
                if constexpr (kQ8) {
                    float lo, hi;
                    unpack2(h[i][k], lo, hi);
                    most = max_nan(most, max_nan(fabsf(lo), fabsf(hi)));
                }
            }
        }
        float lo, hi;
        unpack2(sq, lo, hi);
        const float2 acc = reduce_row<true>(make_float2(lo + hi, most), s[buf]);
        const float r = rsqrtf(acc.x / (float)p.d + p.eps);
        float factor = r;  // y, or y / scale, is (h w) factor
        if (kQ8) {
            float scale = acc.y * r / kE4m3Max;
            factor = kE4m3Max / acc.y;
            if (scale != scale) {  // of NaN in the row or the weight, or of infinity, whose r is zero
                factor = scale;
            } else if (!(scale >= kScaleMin)) {
                scale = kScaleMin;
                factor = fminf(r * (1.f / kScaleMin), 3e38f);
            }
            if (threadIdx.x == 0 && row < p.rows) p.scale[row] = scale;
        }
        const f2 f = pack2(factor, factor);
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int at = place<V>(i, off);
            if (at >= d || at + V <= 0) continue;
#pragma unroll
            for (int k = 0; k < P; k++) h[i][k] = mul2(h[i][k], f);
            if constexpr (!kQ8) {
                store_at<kShift, V>(static_cast<T*>(p.y) + base, at, p.d, h[i]);
            } else {
                unsigned char* q = static_cast<unsigned char*>(p.y) + base;
                float y[V];
                from_pairs<V>(h[i], y);
                if (!kShift || (at >= 0 && at + V <= p.d)) {
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
    float* partial;  // [blocks][d]: each block's sum over its rows of dy h r
};

template <typename T, int kNV, bool kShift>
__global__ void __launch_bounds__(512) ttt_rmsnorm_backward_kernel(const NormBwdParams p) {
    constexpr int V = Elem<T>::kVec, P = V / 2;
    __shared__ float2 s[2][16];
    const long long group = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const long long groups = (long long)gridDim.x * blockDim.y;
    const int off = kShift ? (int)((size_t)group * p.d % V) : 0;
    const T* hp = static_cast<const T*>(p.h) + (size_t)group * p.d;
    const T* gp = static_cast<const T*>(p.dy) + (size_t)group * p.d;
    const T* ip = p.dh_in ? static_cast<const T*>(p.dh_in) + (size_t)group * p.d : nullptr;
    const size_t stride = (size_t)groups * p.d;
    // Rows past 8192 leave no registers for the weight, which waits in shared memory (a thread's own part, 16 bytes
    // side by side with its neighbours'), nor for h and dy in fp32 beside their 16 bits.  The widest variants spill all the
    // same, up to 744 bytes a thread in fp32 and 512 in bf16.
    constexpr bool kWide = kNV * V > 16;
    extern __shared__ ulonglong2 wide[];
    const auto w_place = [&](int i, int k) -> ulonglong2& { return wide[(i * P / 2 + k) * blockDim.x + threadIdx.x]; };
    f2 w[kWide ? 1 : kNV][P], dw[kNV][P];
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int at = place<V>(i, off);
        float v[V];
        f2 wi[P];
#pragma unroll
        for (int k = 0; k < V; k++) v[k] = at + k >= 0 && at + k < p.d ? p.weight[at + k] : 0.f;
        to_pairs<V>(v, wi);
#pragma unroll
        for (int k = 0; k < P / 2; k++) {
            if (kWide) {
                w_place(i, k) = make_ulonglong2(wi[2 * k], wi[2 * k + 1]);
            } else {
                w[kWide ? 0 : i][2 * k] = wi[2 * k];
                w[kWide ? 0 : i][2 * k + 1] = wi[2 * k + 1];
            }
        }
#pragma unroll
        for (int k = 0; k < P; k++) dw[i][k] = pack2(0.f, 0.f);
    }
    // 16-bit rows of up to 8192 leave registers for the next row of h and dy to be on its way (32768 rows of 2048: 95 us against 115)
    constexpr bool kAhead = sizeof(T) == 2 && !kWide, kPastLate = sizeof(T) == 4 && kWide;
    Raw<T, V> rh[kNV], rg[kNV], past[kNV];
    const auto fetch = [&](int d) {
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int at = place<V>(i, off);
            load_at<kShift>(rh[i], hp, at, d);
            load_at<kShift>(rg[i], gp, at, d);
        }
        hp += stride;
        gp += stride;
    };
    if (kAhead) fetch(group < p.rows ? p.d : -V);
    int buf = 0;
    for (long long row = group; row - threadIdx.y < p.rows; row += groups, buf ^= 1) {
        const int d = row < p.rows ? p.d : -V;
        f2 kept_h[kWide ? 1 : kNV][P], kept_dy[kWide ? 1 : kNV][P], sq = pack2(0.f, 0.f), dot = sq;
        if (!kAhead) fetch(d);
        const auto fetch_past = [&] {
            if (!ip) return;
#pragma unroll
            for (int i = 0; i < kNV; i++) load_at<kShift>(past[i], ip, place<V>(i, off), d);
            ip += stride;
        };
        if (!kPastLate) fetch_past();
        if constexpr (!kWide) {
#pragma unroll
            for (int i = 0; i < kNV; i++) {
                pairs_of(rh[i], kept_h[i]);
                pairs_of(rg[i], kept_dy[i]);
            }
            if (kAhead) fetch(row + groups < p.rows ? p.d : -V);
        }
        // the i-th vector of h, dy and the weight
        const auto values = [&](int i, f2(&h)[P], f2(&dy)[P], f2(&wi)[P]) {
            if constexpr (kWide) {
                pairs_of(rh[i], h);
                pairs_of(rg[i], dy);
            }
#pragma unroll
            for (int k = 0; k < P / 2; k++) {
                if constexpr (kWide) {
                    const ulonglong2 a = w_place(i, k);
                    wi[2 * k] = a.x;
                    wi[2 * k + 1] = a.y;
                } else {
#pragma unroll
                    for (int q = 2 * k; q < 2 * k + 2; q++) {
                        h[q] = kept_h[i][q];
                        dy[q] = kept_dy[i][q];
                        wi[q] = w[i][q];
                    }
                }
            }
        };
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            f2 h[P], dy[P], wi[P];
            values(i, h, dy, wi);
#pragma unroll
            for (int k = 0; k < P; k++) {
                sq = fma2(h[k], h[k], sq);
                dot = fma2(mul2(dy[k], wi[k]), h[k], dot);
            }
        }
        float a0, a1, b0, b1;
        unpack2(sq, a0, a1);
        unpack2(dot, b0, b1);
        const float2 acc = reduce_row<false>(make_float2(a0 + a1, b0 + b1), s[buf]);
        const float r = rsqrtf(acc.x / (float)p.d + p.eps);
        const float c = -(acc.y / (float)p.d * r) * r * r;  // in this order: r^3 alone passes the floats' range for tiny and for large rows
        const f2 r2 = pack2(r, r), c2 = pack2(c, c);
        T* out = static_cast<T*>(p.dh) + (size_t)row * p.d;
        if (kPastLate) fetch_past();
        if (kWide && sizeof(T) == 2) {  // the 16 bits are turned into fp32 a second time rather than kept so
#pragma unroll
            for (int i = 0; i < kNV; i++)
#pragma unroll
                for (int k = 0; k < Raw<T, V>::kWords; k++) asm volatile("" : "+r"(rh[i].w[k]), "+r"(rg[i].w[k]));
        }
#pragma unroll
        for (int i = 0; i < kNV; i++) {
            const int at = place<V>(i, off);
            f2 o[P], h[P], dy[P], wi[P];
            values(i, h, dy, wi);
            if (ip)
                pairs_of(past[i], o);
            else
#pragma unroll
                for (int k = 0; k < P; k++) o[k] = pack2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < P; k++) {
                o[k] = fma2(c2, h[k], o[k]);
                const f2 rdy = mul2(r2, dy[k]);
                o[k] = fma2(rdy, wi[k], o[k]);
                dw[i][k] = fma2(rdy, h[k], dw[i][k]);
            }
            if (at < d && at + V > 0) store_at<kShift, V>(out, at, d, o);
        }
    }
    // rows of a block that are side by side (d at most 16 elements of 32 lanes) are added up first
    __shared__ float sums[128 * 16];
    float* part = blockDim.y > 1 ? sums + threadIdx.y * p.d : p.partial + (size_t)blockIdx.x * p.d;
#pragma unroll
    for (int i = 0; i < kNV; i++) {
        const int at = place<V>(i, off);
        float v[V];
        from_pairs<V>(dw[i], v);
#pragma unroll
        for (int k = 0; k < V; k++)
            if (at + k >= 0 && at + k < p.d) part[at + k] = v[k];
    }
    if (blockDim.y > 1) {
        __syncthreads();
        for (int j = threadIdx.y * blockDim.x + threadIdx.x; j < p.d; j += blockDim.x * blockDim.y) {
            float a = 0.f;
            for (int y = 0; y < (int)blockDim.y; y++) a += sums[y * p.d + j];
            p.partial[(size_t)blockIdx.x * p.d + j] = a;
        }
    }
}

struct Shape {
    int threads_x, threads_y, nv;
    long long blocks;
};

// Threads a row: those that hold it in `nv` vectors each, nv = 16 elements (one vector where a warp or a part
// of one then holds the row, half as many again or twice as many where 512 threads would not).  Rows of a warp or less share a block of
// 128 threads.  Blocks: `resident` threads on each of 148 SMs, or as many as there are rows; where rows start
// inside a vector, rounded down to a multiple of 8.
Shape shape_of(long long rows, int d, int es, int resident) {
    const int v = 16 / es, vecs = d % v == 0 ? d / v : (d + 2 * v - 2) / v, usual = 16 / v;
    Shape s{1, 1, 1, 0};
    if (vecs <= 32) {
        while (s.threads_x < vecs) s.threads_x *= 2;
    } else {
        s.nv = vecs <= 512 * usual ? usual : vecs <= 768 * usual ? 3 * usual / 2 : vecs <= 1024 * usual ? 2 * usual : 2 * usual + 1;
        s.threads_x = ((vecs + s.nv - 1) / s.nv + 31) / 32 * 32;
    }
    if (s.threads_x <= 32) s.threads_y = 128 / s.threads_x;
    const int a_block = s.threads_x * s.threads_y;
    s.blocks = 148LL * (a_block < resident ? resident / a_block : 1);
    if (d % v != 0) s.blocks -= s.blocks % 8;
    const long long need = (rows + s.threads_y - 1) / s.threads_y;
    if (s.blocks > need) s.blocks = need;  // a group then has one row at most
    return s;
}
Shape forward_shape(long long rows, int d, int es) { return shape_of(rows, d, es, 1024); }
Shape backward_shape(long long rows, int d, int es) { return shape_of(rows, d, es, 512); }

// f(vectors a thread, whether rows start inside a vector)
template <typename T, typename F>
cudaError_t by_vectors(int nv, int d, F f) {
    constexpr int kV = Elem<T>::kVec, kUsual = 16 / kV;
    const auto with = [&](auto n) {
        if (d % kV)
            f(n, std::true_type{});
        else
            f(n, std::false_type{});
        return cudaPeekAtLastError();
    };
    if (nv == 1) return with(std::integral_constant<int, 1>{});
    if (nv == kUsual) return with(std::integral_constant<int, kUsual>{});
    if (nv == 3 * kUsual / 2) return with(std::integral_constant<int, 3 * kUsual / 2>{});
    if (nv == 2 * kUsual) return with(std::integral_constant<int, 2 * kUsual>{});
    if (nv == 2 * kUsual + 1) return with(std::integral_constant<int, 2 * kUsual + 1>{});
    return cudaErrorInvalidValue;
}

template <typename T, bool kQ8>
cudaError_t launch_forward(const NormParams& p, cudaStream_t stream) {
    const Shape s = forward_shape(p.rows, p.d, sizeof(T));
    const dim3 block(s.threads_x, s.threads_y);
    return by_vectors<T>(s.nv, p.d, [&](auto nv, auto shift) {
        ttt_rmsnorm_kernel<T, decltype(nv)::value, decltype(shift)::value, kQ8><<<(unsigned)s.blocks, block, 0, stream>>>(p);
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
#pragma unroll 8
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
    cudaError_t e = by_vectors<T>(s.nv, p.d, [&](auto nv, auto shift) {
        const auto kernel = ttt_rmsnorm_backward_kernel<T, decltype(nv)::value, decltype(shift)::value>;
        constexpr int kBytes = decltype(nv)::value * 16 / (int)sizeof(T) * 4;  // of the weight, a thread
        const int smem = kBytes > 64 ? kBytes * s.threads_x : 0;
        if (smem > 48 * 1024 - 8192 - 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        kernel<<<(unsigned)s.blocks, block, smem, stream>>>(p);
    });
    if (e != cudaSuccess) return e;
    return launch_column_sum((int)s.blocks, p.d, p.partial, dweight, stream);
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
    return (size_t)s.blocks * d * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, float* workspace, cudaStream_t stream) {
    const NormBwdParams p{(long long)a.B * a.T, a.d, a.eps, a.h, a.dy, a.dh_in, a.weight, a.dh, workspace};
    return a.dtype == TTT_BF16 ? launch_backward<__nv_bfloat16>(p, a.dweight, stream)
                               : launch_backward<float>(p, a.dweight, stream);
}

}  // namespace ttt
