// Short causal depthwise convolution of token rows with an optional SiLU, forward (prompts, padded
// batches, a carried state; single tokens in place) and backward.
//
//   p_t = bias + sum_{j < W} w_j x_{t - (W - 1) + j},   y_t = silu(p_t) or p_t
// per channel; rows before the first token are the state's (the last W - 1 rows of what came before) or
// zero.  Backward, with dp_t = dy_t act'(p_t):
//   dx_t = sum_j w_j dp_{t + W - 1 - j},  dw_j = sum_t dp_t x_{t - (W - 1) + j},  dbias = sum_t dp_t
// and the gradient of the last W - 1 rows gets that of the final state added.
//
// Bound by HBM (forward: a row read and a row written).  A thread owns V = 4 neighbouring channels (1
// where rows do not allow it) and walks a piece of the tokens with the last W - 1 rows in registers and
// the next rows on their way, so a row is read once but for the W - 1 rows before each piece.  Sums are in
// fp32, rounded once.
//
// Measured (width 4, bf16): forward of 2 x 32768 x 2048, x half of a wider projection's rows, 104 us, 5.2 TB/s, 0.78 of the
// copy bandwidth; the SiLUs' special functions take 58 % of their pipe beside it.  Rows fetched one by one as a place came
// free, instead of four at a time, took 209 us.  Gradient of 8 x 2048 x 1536: 57 us, 2.6 TB/s; four channels'
// dw and dbias beside the window leave registers for few rows on their way, some 21 KB an SM, and more, shorter pieces
// took 62 us.  In fp32 the forward of 32768 x 2048 takes 92 us (0.89) and the gradient of 8 x 2048 x 1536 125 us; a row
// takes twice the registers there, and the variants of width 3 and 4 spill up to 236 and 508 bytes a thread.
#include "block_internal.h"
#include "vec_io.cuh"

#include <type_traits>

namespace ttt {
namespace {

__device__ __forceinline__ int length_of(const int* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

struct ConvParams {
    int T, C, piece, pieces, groups;  // groups: channel groups (blocks) a row
    long long strips;                 // B pieces: what a thread walks of its channels
    long long ld;                     // elements from one row of x to the next
    const void *x, *state0;
    const float *weight, *bias;
    const int* lengths;
    void *y, *state_T;
};

constexpr int kThreads = 128;
constexpr int kAhead = 4;  // rows on their way while the four before them are worked on

// Blocks are kThreads columns (of one or four channels) of one strip, or of several where a row has fewer (kNarrow:
// piece and sequence then differ from thread to thread, which costs registers that wide rows have no use for).
inline dim3 block_of(int columns, bool narrow) {
    int x = kThreads;
    while (narrow && x > 8 && x / 2 >= columns) x /= 2;
    return dim3(x, kThreads / x);
}
struct Place {
    int column, piece, b;
    bool on;
};
template <bool kNarrow>
__device__ __forceinline__ Place place_of(int groups, int pieces, long long strips) {
    const int grp = (int)(blockIdx.x % groups);
    long long strip = blockIdx.x / groups;
    if constexpr (kNarrow) strip = strip * blockDim.y + threadIdx.y;
    Place at;
    at.column = grp * (kNarrow ? (int)blockDim.x : kThreads) + (int)threadIdx.x;
    at.on = !kNarrow || strip < strips;
    at.piece = (int)(strip % pieces);
    at.b = (int)(strip / pieces);
    return at;
}

// Row t of the window of sequence b (t < 0: the state's rows), the thread's channels.
template <typename T, int V, int W>
__device__ __forceinline__ void window_row(const T* x, const T* state, long long ld, int C, int t, float (&v)[V]) {
    if (t >= 0) {
        load_vec<V>(x + (long long)t * ld, v);
    } else if (state) {
        load_vec<V>(state + (long long)(t + W - 1) * C, v);
    } else {
#pragma unroll
        for (int k = 0; k < V; k++) v[k] = 0.f;
    }
}

// The taps of V neighbouring channels: V W floats side by side
template <int V, int W>
__device__ __forceinline__ void load_taps(const float* weight, int c, f2 (&w)[W][(V + 1) / 2]) {
    float v[V * W];
    if constexpr (V * W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V * W / 4; i++) {
            const float4 r = reinterpret_cast<const float4*>(weight + (size_t)c * W)[i];
            v[4 * i] = r.x;
            v[4 * i + 1] = r.y;
            v[4 * i + 2] = r.z;
            v[4 * i + 3] = r.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; i++) v[i] = weight[(size_t)c * W + i];
    }
#pragma unroll
    for (int j = 0; j < W; j++) {
        float tap[V];
#pragma unroll
        for (int k = 0; k < V; k++) tap[k] = v[k * W + j];
        to_pairs<V>(tap, w[j]);
    }
}
template <int V>
__device__ __forceinline__ void load_bias(const float* bias, int c, f2 (&o)[(V + 1) / 2]) {
    float v[V];
#pragma unroll
    for (int k = 0; k < V; k++) v[k] = bias ? bias[c + k] : 0.f;
    to_pairs<V>(v, o);
}

// bias + sum_j w_j x: the window's rows, then the newest
template <int W, int P>
__device__ __forceinline__ void taps(const f2 (&w)[W][P], const f2 (&bias)[P], const f2 (&win)[W - 1][P], const f2 (&in)[P],
                                     f2 (&a)[P]) {
#pragma unroll
    for (int k = 0; k < P; k++) {
        a[k] = fma2(w[0][k], win[0][k], bias[k]);
#pragma unroll
        for (int j = 1; j < W - 1; j++) a[k] = fma2(w[j][k], win[j][k], a[k]);
        a[k] = fma2(w[W - 1][k], in[k], a[k]);
    }
}
template <int W, int P>
__device__ __forceinline__ void shift_in(f2 (&win)[W - 1][P], const f2 (&in)[P]) {
#pragma unroll
    for (int k = 0; k < P; k++) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; j++) win[j][k] = win[j + 1][k];
        win[W - 2][k] = in[k];
    }
}

template <typename T, int V, int W, bool kSilu, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 6) ttt_conv_kernel(const ConvParams p) {
    constexpr int P = (V + 1) / 2;  // pairs
    const Place at = place_of<kNarrow>(p.groups, p.pieces, p.strips);
    const int piece = at.piece, b = at.b, c = at.column * V;
    if (c >= p.C || !at.on) return;
    const int n = length_of(p.lengths, b, p.T);
    const T* x = static_cast<const T*>(p.x) + (long long)b * p.T * p.ld + c;
    const T* state = p.state0 ? static_cast<const T*>(p.state0) + (long long)b * (W - 1) * p.C + c : nullptr;
    T* y = static_cast<T*>(p.y) + (long long)b * p.T * p.C + c;

    const int t0 = piece * p.piece, t1 = min(t0 + p.piece, p.T);
    const int live = min(t1, n);
    // Two batches of rows: one on its way while the other is worked on.  (A batch is loaded as a whole: a
    // load into a slot just used up would have to be waited for together with the oldest one.)
    Raw<T, V> rows[2][kAhead];
    const auto load = [&](Raw<T, V>(&to)[kAhead], int t) {
#pragma unroll
        for (int r = 0; r < kAhead; r++)
            if (t + r < live) to[r].load(x + (long long)(t + r) * p.ld);
    };
    load(rows[0], t0);
    f2 w[W][P], bias[P], win[W - 1][P];
    load_bias<V>(p.bias, c, bias);
    load_taps<V, W>(p.weight, c, w);
    if (t0 < live) {
#pragma unroll
        for (int i = 0; i < W - 1; i++) {
            float v[V];
            window_row<T, V, W>(x, state, p.ld, p.C, t0 - (W - 1) + i, v);
            to_pairs<V>(v, win[i]);
        }
    }
    // The final state, by the threads of the first piece, who alone read state0: it may be written in
    // place.  They have what they need of it in `win` (t0 = 0) or read it here before they write.
    if (piece == 0 && p.state_T) {
        float last[W - 1][V];
#pragma unroll
        for (int i = 0; i < W - 1; i++) window_row<T, V, W>(x, state, p.ld, p.C, n - (W - 1) + i, last[i]);
        T* out = static_cast<T*>(p.state_T) + (long long)b * (W - 1) * p.C + c;
#pragma unroll
        for (int i = 0; i < W - 1; i++) store_vec<V>(out + (long long)i * p.C, last[i]);
    }
    const auto work = [&](const Raw<T, V>(&from)[kAhead], int t, auto whole) {
#pragma unroll
        for (int r = 0; r < kAhead; r++) {
            if (!decltype(whole)::value && t + r >= live) break;
            float v[V];
            f2 in[P], a[P];
            from[r].get(v);
            to_pairs<V>(v, in);
            taps<W, P>(w, bias, win, in, a);
            shift_in<W, P>(win, in);
            if constexpr (kSilu)
#pragma unroll
                for (int k = 0; k < P; k++) a[k] = mul2(a[k], sigmoid2(a[k]));
            from_pairs<V>(a, v);
            store_vec<V>(y + (long long)(t + r) * p.C, v);
        }
    };
    int t = t0;
    for (; t + 2 * kAhead <= live; t += 2 * kAhead) {
        load(rows[1], t + kAhead);
        work(rows[0], t, std::true_type{});
        load(rows[0], t + 2 * kAhead);
        work(rows[1], t + kAhead, std::true_type{});
    }
    if (t < live) {
        load(rows[1], t + kAhead);
        work(rows[0], t, std::false_type{});
        work(rows[1], t + kAhead, std::false_type{});
    }
    float zero[V];
#pragma unroll
    for (int k = 0; k < V; k++) zero[k] = 0.f;
    for (t = max(t0, n); t < t1; t++) store_vec<V>(y + (long long)t * p.C, zero);
}

struct ConvBwdParams {
    int T, C, piece, pieces, groups;
    long long strips, ld;
    const void *x, *state0, *dy, *dstate_T;
    const float *weight, *bias;
    const int* lengths;
    void *dx, *dstate0;
    float* partial;  // [B][pieces][W + 1][C]
};

constexpr int kBack = 4;     // rows of x and dy on their way
constexpr int kBackVec = 4;  // channels a thread, where rows allow it

template <typename T, int V, int W, bool kSilu, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 4) ttt_conv_backward_kernel(const ConvBwdParams p) {
    constexpr int P = (V + 1) / 2;
    const Place at = place_of<kNarrow>(p.groups, p.pieces, p.strips);
    const int piece = at.piece, b = at.b, c = at.column * V;
    if (c >= p.C || !at.on) return;
    const int n = length_of(p.lengths, b, p.T);

    const f2 zero2 = pack2(0.f, 0.f), one2 = pack2(1.f, 1.f);
    f2 dw[W][P], db[P];
#pragma unroll
    for (int k = 0; k < P; k++) {
        db[k] = zero2;
#pragma unroll
        for (int j = 0; j < W; j++) dw[j][k] = zero2;
    }
    // This piece: the gradients of rows [r0, t1) of the window, which for the first piece begins W - 1 rows
    // before token 0 (the state's rows).  Row t needs dp_t .. dp_{t + W - 1}; dp of the piece's own tokens
    // counts for dw.
    const int t0 = piece * p.piece, t1 = min(t0 + p.piece, p.T);
    {
        const T* x = static_cast<const T*>(p.x) + (long long)b * p.T * p.ld + c;
        const T* state = p.state0 ? static_cast<const T*>(p.state0) + (long long)b * (W - 1) * p.C + c : nullptr;
        const T* dy = static_cast<const T*>(p.dy) + (long long)b * p.T * p.C + c;
        const T* dst = p.dstate_T ? static_cast<const T*>(p.dstate_T) + (long long)b * (W - 1) * p.C + c : nullptr;
        T* dx = static_cast<T*>(p.dx) + (long long)b * p.T * p.C + c;
        T* ds0 = p.dstate0 ? static_cast<T*>(p.dstate0) + (long long)b * (W - 1) * p.C + c : nullptr;
        const int r0 = t0 == 0 ? -(W - 1) : t0, stop = t1 + W - 1, live = min(stop, n);
        Raw<T, V> rows[2][kBack], grads[2][kBack];
        const auto load = [&](int which, int t) {
#pragma unroll
            for (int q = 0; q < kBack; q++)
                if (t + q < live) {
                    rows[which][q].load(x + (long long)(t + q) * p.ld);
                    grads[which][q].load(dy + (long long)(t + q) * p.C);
                }
        };
        load(0, t0);
        f2 w[W][P], bias[P], win[W - 1][P], dp[W - 1][P];
        load_bias<V>(p.bias, c, bias);
        load_taps<V, W>(p.weight, c, w);
#pragma unroll
        for (int i = 0; i < W - 1; i++) {
#pragma unroll
            for (int k = 0; k < P; k++) dp[i][k] = win[i][k] = zero2;
            if (t0 < live) {
                float v[V];
                window_row<T, V, W>(x, state, p.ld, p.C, t0 - (W - 1) + i, v);
                to_pairs<V>(v, win[i]);
            }
        }
        // Step t: dp_t is computed, and with it row t - (W - 1) is complete.  `inside`: both are tokens of the piece.
        const auto step = [&](int t, const Raw<T, V>& row, const Raw<T, V>& grad, auto inside) {
            constexpr bool kInside = decltype(inside)::value;
            f2 now[P];
#pragma unroll
            for (int k = 0; k < P; k++) now[k] = zero2;
            if (kInside || t < live) {
                float v[V];
                f2 in[P];
                row.get(v);
                to_pairs<V>(v, in);
                grad.get(v);
                to_pairs<V>(v, now);
                if constexpr (kSilu) {
                    f2 a[P];
                    taps<W, P>(w, bias, win, in, a);
#pragma unroll
                    for (int k = 0; k < P; k++) {  // dy s (1 + a (1 - s))
                        const f2 sg = sigmoid2(a[k]);
                        const f2 rest = fma2(sg, pack2(-1.f, -1.f), one2);
                        now[k] = mul2(mul2(now[k], sg), fma2(a[k], rest, one2));
                    }
                }
                if (kInside || t < t1) {
#pragma unroll
                    for (int k = 0; k < P; k++) {
                        db[k] = add2(db[k], now[k]);
#pragma unroll
                        for (int j = 0; j < W - 1; j++) dw[j][k] = fma2(now[k], win[j][k], dw[j][k]);
                        dw[W - 1][k] = fma2(now[k], in[k], dw[W - 1][k]);
                    }
                }
                shift_in<W, P>(win, in);
            }
            const int r = t - (W - 1);  // the row that is complete
            f2 o2[P];
            float o[V];
#pragma unroll
            for (int k = 0; k < P; k++) {
                o2[k] = mul2(w[0][k], now[k]);
#pragma unroll
                for (int j = 1; j < W; j++) o2[k] = fma2(w[j][k], dp[W - 1 - j][k], o2[k]);
            }
            from_pairs<V>(o2, o);
            if constexpr (kInside) {
                store_vec<V>(dx + (long long)r * p.C, o);
            } else if (r >= r0) {
                const int i = t - n;  // its place in the final state
                if (dst && i >= 0 && i < W - 1) {
                    float add[V];
                    load_vec<V>(dst + (long long)i * p.C, add);
#pragma unroll
                    for (int k = 0; k < V; k++) o[k] += add[k];
                }
                if (r >= 0)
                    store_vec<V>(dx + (long long)r * p.C, o);
                else if (ds0)
                    store_vec<V>(ds0 + (long long)(r + W - 1) * p.C, o);
            }
            shift_in<W, P>(dp, now);
        };
        for (int tb = t0; tb < stop; tb += 2 * kBack) {
            load(1, tb + kBack);
            if (tb - (W - 1) >= t0 && tb + 2 * kBack <= min(t1, n)) {
#pragma unroll
                for (int q = 0; q < kBack; q++) step(tb + q, rows[0][q], grads[0][q], std::true_type{});
                load(0, tb + 2 * kBack);
#pragma unroll
                for (int q = 0; q < kBack; q++) step(tb + kBack + q, rows[1][q], grads[1][q], std::true_type{});
            } else {
#pragma unroll
                for (int q = 0; q < kBack; q++)
                    if (tb + q < stop) step(tb + q, rows[0][q], grads[0][q], std::false_type{});
                load(0, tb + 2 * kBack);
#pragma unroll
                for (int q = 0; q < kBack; q++)
                    if (tb + kBack + q < stop) step(tb + kBack + q, rows[1][q], grads[1][q], std::false_type{});
            }
        }
    }
    float* part = p.partial + (((size_t)b * p.pieces + piece) * (W + 1)) * p.C + c;
#pragma unroll
    for (int j = 0; j <= W; j++) {
        float v[V];
        from_pairs<V>(j < W ? dw[j % W] : db, v);
        store_vec<V>(part + (size_t)j * p.C, v);
    }
}

// dweight [C][W] and dbias [C] from the pieces' partials [rows][W + 1][C]: 32 channels and one tap a
// block, 32 threads a sum.  The order of the additions goes by the shape alone.
__global__ void __launch_bounds__(1024) ttt_conv_weight_sum_kernel(int rows, int W, int C, const float* __restrict__ partial,
                                                                   float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y;
    float a = 0.f;
    if (c < C)
#pragma unroll 8
        for (int r = threadIdx.y; r < rows; r += 32) a += partial[((size_t)r * (W + 1) + j) * C + c];
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 32; i++) a += s[i][threadIdx.x];
        if (j < W)
            dweight[(size_t)c * W + j] = a;
        else if (dbias)
            dbias[c] = a;
    }
}

bool rows_aligned(const void* p, long long ld, int bytes, int es) {
    return !p || ((reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (ld * es) % bytes == 0);
}

template <typename F>
cudaError_t by_width(int W, int silu, F f) {
    const auto with = [&](auto w) {
        if (silu)
            f(w, std::true_type{});
        else
            f(w, std::false_type{});
    };
    switch (W) {
        case 2: with(std::integral_constant<int, 2>{}); break;
        case 3: with(std::integral_constant<int, 3>{}); break;
        case 4: with(std::integral_constant<int, 4>{}); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaPeekAtLastError();
}

// Tokens a thread walks: 64, halved down to 4 while the launch has fewer threads than 148 SMs hold.
// Never under W - 1 = 3, so that only the first piece reads the state.
int forward_piece(const ConvArgs& a, int vec) {
    const long long columns = (long long)a.B * ((a.C + vec - 1) / vec);
    int piece = 64;
    while (piece > 4 && columns * ((a.T + piece - 1) / piece) < 148LL * 2048) piece /= 2;
    return piece;
}

template <typename T>
cudaError_t forward(const ConvArgs& a, cudaStream_t stream) {
    constexpr int kV = 4;
    const bool vec = a.C % kV == 0 && rows_aligned(a.x, a.ld, kV * sizeof(T), sizeof(T));
    const int v = vec ? kV : 1;
    ConvParams p{};
    p.T = a.T;
    p.C = a.C;
    p.piece = forward_piece(a, v);
    p.pieces = a.T > 0 ? (a.T + p.piece - 1) / p.piece : 1;  // an empty sequence still passes its state on
    const int columns = (a.C + v - 1) / v;
    const bool narrow = columns <= kThreads / 2;
    const dim3 threads = block_of(columns, narrow);
    p.groups = (columns + threads.x - 1) / threads.x;
    p.strips = (long long)a.B * p.pieces;
    p.ld = a.ld;
    p.x = a.x;
    p.state0 = a.state0;
    p.weight = a.weight;
    p.bias = a.bias;
    p.lengths = a.lengths;
    p.y = a.y;
    p.state_T = a.state_T;
    const long long blocks = (p.strips + threads.y - 1) / threads.y * p.groups;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    return by_width(a.W, a.silu, [&](auto w, auto silu) {
        constexpr int W = decltype(w)::value;
        constexpr bool kSilu = decltype(silu)::value;
        const auto start = [&](auto kernel) { kernel<<<(unsigned)blocks, threads, 0, stream>>>(p); };
        if (vec)
            narrow ? start(ttt_conv_kernel<T, kV, W, kSilu, true>) : start(ttt_conv_kernel<T, kV, W, kSilu, false>);
        else
            narrow ? start(ttt_conv_kernel<T, 1, W, kSilu, true>) : start(ttt_conv_kernel<T, 1, W, kSilu, false>);
    });
}

// Tokens a thread of the backward walks: 128, halved down to 16 while the launch has fewer than 256 threads for
// each of 148 SMs.  The width of a block counts for DRAM: 128 threads side by side read 1 KB of a row, where 32
// with their four warps at four places of the sequence took 1.4 times as long.
int backward_piece(int B, int T, int C, int vec) {
    const long long columns = (long long)B * ((C + vec - 1) / vec);
    int piece = 128;
    while (piece > 16 && columns * ((T + piece - 1) / piece) < 148LL * 256) piece /= 2;
    return piece;
}

template <typename T>
cudaError_t backward(const ConvBwdArgs& a, float* workspace, cudaStream_t stream) {
    constexpr int kV = kBackVec;
    const bool vec = a.f.C % kV == 0 && rows_aligned(a.f.x, a.f.ld, kV * sizeof(T), sizeof(T));
    const int v = vec ? kV : 1;
    ConvBwdParams p{};
    p.T = a.f.T;
    p.C = a.f.C;
    p.piece = backward_piece(a.f.B, a.f.T, a.f.C, v);
    p.pieces = a.f.T > 0 ? (a.f.T + p.piece - 1) / p.piece : 1;
    const int columns = (a.f.C + v - 1) / v;
    const bool narrow = columns <= kThreads / 2;
    const dim3 threads = block_of(columns, narrow);
    p.groups = (columns + threads.x - 1) / threads.x;
    p.strips = (long long)a.f.B * p.pieces;
    p.ld = a.f.ld;
    p.x = a.f.x;
    p.state0 = a.f.state0;
    p.dy = a.dy;
    p.dstate_T = a.dstate_T;
    p.weight = a.f.weight;
    p.bias = a.f.bias;
    p.lengths = a.f.lengths;
    p.dx = a.dx;
    p.dstate0 = a.dstate0;
    p.partial = workspace;
    const long long blocks = (p.strips + threads.y - 1) / threads.y * p.groups;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    cudaError_t e = by_width(a.f.W, a.f.silu, [&](auto w, auto silu) {
        constexpr int W = decltype(w)::value;
        constexpr bool kSilu = decltype(silu)::value;
        const auto start = [&](auto kernel) { kernel<<<(unsigned)blocks, threads, 0, stream>>>(p); };
        if (vec)
            narrow ? start(ttt_conv_backward_kernel<T, kV, W, kSilu, true>) : start(ttt_conv_backward_kernel<T, kV, W, kSilu, false>);
        else
            narrow ? start(ttt_conv_backward_kernel<T, 1, W, kSilu, true>) : start(ttt_conv_backward_kernel<T, 1, W, kSilu, false>);
    });
    if (e != cudaSuccess) return e;
    ttt_conv_weight_sum_kernel<<<dim3((a.f.C + 31) / 32, a.f.W + 1), dim3(32, 32), 0, stream>>>(
        a.f.B * p.pieces, a.f.W, a.f.C, workspace, a.dweight, a.dbias);
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, cudaStream_t stream) {
    return a.dtype == TTT_BF16 ? forward<__nv_bfloat16>(a, stream) : forward<float>(a, stream);
}

size_t conv_backward_workspace_bytes(int B, int T, int C, int W) {
    if (B < 1 || T < 0 || C < 1 || W < 2 || W > kConvMaxWidth) return 0;
    // the launch picks four channels a thread, or one where alignment asks for it: room for either
    size_t most = 0;
    for (int v : {1, kBackVec}) {
        const int piece = backward_piece(B, T, C, v);
        const size_t pieces = T > 0 ? (T + piece - 1) / piece : 1;
        const size_t bytes = (size_t)B * pieces * (W + 1) * C * sizeof(float);
        if (bytes > most) most = bytes;
    }
    return most;
}

cudaError_t launch_conv_backward(const ConvBwdArgs& a, float* workspace, cudaStream_t stream) {
    return a.f.dtype == TTT_BF16 ? backward<__nv_bfloat16>(a, workspace, stream) : backward<float>(a, workspace, stream);
}

}  // namespace ttt
