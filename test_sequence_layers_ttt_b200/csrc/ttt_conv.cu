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
#include "block_internal.h"
#include "vec_io.cuh"

namespace ttt {
namespace {

__device__ __forceinline__ int length_of(const int* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

struct ConvParams {
    int T, C, piece, pieces, groups;  // groups: channel groups (blocks) a row
    long long ld;                     // elements from one row of x to the next
    const void *x, *state0;
    const float *weight, *bias;
    const int* lengths;
    void *y, *state_T;
    int silu;
};

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // rows on their way while the ones before them are worked on

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

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) ttt_conv_kernel(const ConvParams p) {
    const long long block = blockIdx.x;
    const int grp = (int)(block % p.groups);
    const int piece = (int)(block / p.groups % p.pieces);
    const int b = (int)(block / p.groups / p.pieces);
    const int c = (grp * kThreads + threadIdx.x) * V;
    if (c >= p.C) return;
    const int n = length_of(p.lengths, b, p.T);
    const T* x = static_cast<const T*>(p.x) + (long long)b * p.T * p.ld + c;
    const T* state = p.state0 ? static_cast<const T*>(p.state0) + (long long)b * (W - 1) * p.C + c : nullptr;
    T* y = static_cast<T*>(p.y) + (long long)b * p.T * p.C + c;

    float w[W][V], bias[V], win[W - 1][V];
#pragma unroll
    for (int k = 0; k < V; k++) {
        bias[k] = p.bias ? p.bias[c + k] : 0.f;
#pragma unroll
        for (int j = 0; j < W; j++) w[j][k] = p.weight[(size_t)(c + k) * W + j];
    }
    const int t0 = piece * p.piece, t1 = min(t0 + p.piece, p.T);
    const int live = min(t1, n);
    if (t0 < live) {
#pragma unroll
        for (int i = 0; i < W - 1; i++) window_row<T, V, W>(x, state, p.ld, p.C, t0 - (W - 1) + i, win[i]);
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
    Raw<T, V> next[kAhead];
#pragma unroll
    for (int r = 0; r < kAhead; r++)
        if (t0 + r < live) next[r].load(x + (long long)(t0 + r) * p.ld);
    int t = t0;
    for (; t < live; t += kAhead) {
#pragma unroll
        for (int r = 0; r < kAhead; r++) {
            if (t + r < live) {
                float in[V], o[V];
                next[r].get(in);
                if (t + kAhead + r < live) next[r].load(x + (long long)(t + kAhead + r) * p.ld);
#pragma unroll
                for (int k = 0; k < V; k++) {
                    float a = bias[k];
#pragma unroll
                    for (int j = 0; j < W - 1; j++) a += w[j][k] * win[j][k];
                    a += w[W - 1][k] * in[k];
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; j++) win[j][k] = win[j + 1][k];
                    win[W - 2][k] = in[k];
                    o[k] = p.silu ? a * sigmoid(a) : a;
                }
                store_vec<V>(y + (long long)(t + r) * p.C, o);
            }
        }
    }
    float zero[V];
#pragma unroll
    for (int k = 0; k < V; k++) zero[k] = 0.f;
    for (t = max(t0, n); t < t1; t++) store_vec<V>(y + (long long)t * p.C, zero);
}

struct ConvBwdParams {
    int T, C, piece, pieces, groups;
    long long ld;
    const void *x, *state0, *dy, *dstate_T;
    const float *weight, *bias;
    const int* lengths;
    void *dx, *dstate0;
    float* partial;  // [B][pieces][W + 1][C]
    int silu;
};

constexpr int kBack = 4;  // rows of x and dy on their way
constexpr int kLanes = 32, kSub = 4;  // threads: 32 channel vectors x 4 runs of a piece's tokens

template <typename T, int V, int W>
__global__ void __launch_bounds__(kLanes * kSub) ttt_conv_backward_kernel(const ConvBwdParams p) {
    __shared__ float s[kSub][W + 1][kLanes * V];
    const long long block = blockIdx.x;
    const int grp = (int)(block % p.groups);
    const int piece = (int)(block / p.groups % p.pieces);
    const int b = (int)(block / p.groups / p.pieces);
    const int c = (grp * kLanes + threadIdx.x) * V;
    const bool on = c < p.C;
    const int n = length_of(p.lengths, b, p.T);

    float dw[W][V], db[V];
#pragma unroll
    for (int k = 0; k < V; k++) {
        db[k] = 0.f;
#pragma unroll
        for (int j = 0; j < W; j++) dw[j][k] = 0.f;
    }
    if (on) {
        const T* x = static_cast<const T*>(p.x) + (long long)b * p.T * p.ld + c;
        const T* state = p.state0 ? static_cast<const T*>(p.state0) + (long long)b * (W - 1) * p.C + c : nullptr;
        const T* dy = static_cast<const T*>(p.dy) + (long long)b * p.T * p.C + c;
        const T* dst = p.dstate_T ? static_cast<const T*>(p.dstate_T) + (long long)b * (W - 1) * p.C + c : nullptr;
        T* dx = static_cast<T*>(p.dx) + (long long)b * p.T * p.C + c;
        T* ds0 = p.dstate0 ? static_cast<T*>(p.dstate0) + (long long)b * (W - 1) * p.C + c : nullptr;
        float w[W][V], bias[V], win[W - 1][V], dp[W - 1][V];
#pragma unroll
        for (int k = 0; k < V; k++) {
            bias[k] = p.bias ? p.bias[c + k] : 0.f;
#pragma unroll
            for (int j = 0; j < W; j++) w[j][k] = p.weight[(size_t)(c + k) * W + j];
        }
        // This run: the gradients of rows [r0, r1) of the window, which for the first run begins W - 1
        // rows before token 0 (the state's rows).  Row t needs dp_t .. dp_{t + W - 1}; dp of the run's
        // own tokens counts for dw.
        const int run = p.piece / kSub;
        const int t0 = piece * p.piece + (int)threadIdx.y * run, t1 = min(t0 + run, p.T);
        const int r0 = t0 == 0 ? -(W - 1) : t0;
#pragma unroll
        for (int i = 0; i < W - 1; i++) {
#pragma unroll
            for (int k = 0; k < V; k++) dp[i][k] = win[i][k] = 0.f;
            if (t0 < t1 && t0 < n) window_row<T, V, W>(x, state, p.ld, p.C, t0 - (W - 1) + i, win[i]);
        }
        // step t: dp_t is computed, and with it row t - (W - 1) is complete
        if (t0 < t1 || (t0 == 0 && p.T == 0)) {
            const int stop = t1 + W - 1, live = min(stop, n);
            Raw<T, V> next_x[kBack], next_g[kBack];
#pragma unroll
            for (int q = 0; q < kBack; q++)
                if (t0 + q < live) {
                    next_x[q].load(x + (long long)(t0 + q) * p.ld);
                    next_g[q].load(dy + (long long)(t0 + q) * p.C);
                }
            for (int tq = t0; tq < stop; tq += kBack)
#pragma unroll
            for (int q = 0; q < kBack; q++) {
                const int t = tq + q;
                if (t >= stop) break;
                float now[V];
#pragma unroll
                for (int k = 0; k < V; k++) now[k] = 0.f;
                if (t < live) {
                    float in[V], g[V];
                    next_x[q].get(in);
                    next_g[q].get(g);
                    if (t + kBack < live) {
                        next_x[q].load(x + (long long)(t + kBack) * p.ld);
                        next_g[q].load(dy + (long long)(t + kBack) * p.C);
                    }
#pragma unroll
                    for (int k = 0; k < V; k++) {
                        float a = bias[k];
#pragma unroll
                        for (int j = 0; j < W - 1; j++) a += w[j][k] * win[j][k];
                        a += w[W - 1][k] * in[k];
                        const float sg = sigmoid(a);
                        now[k] = p.silu ? g[k] * sg * (1.f + a * (1.f - sg)) : g[k];
                        if (t < t1) {
                            db[k] += now[k];
#pragma unroll
                            for (int j = 0; j < W - 1; j++) dw[j][k] += now[k] * win[j][k];
                            dw[W - 1][k] += now[k] * in[k];
                        }
#pragma unroll
                        for (int j = 0; j + 1 < W - 1; j++) win[j][k] = win[j + 1][k];
                        win[W - 2][k] = in[k];
                    }
                }
                const int r = t - (W - 1);  // the row that is complete
                if (r >= r0) {
                    float o[V], add[V];
#pragma unroll
                    for (int k = 0; k < V; k++) add[k] = 0.f;
                    const int i = r + (W - 1) - n;  // its place in the final state
                    if (dst && i >= 0 && i < W - 1) load_vec<V>(dst + (long long)i * p.C, add);
#pragma unroll
                    for (int k = 0; k < V; k++) {
                        float a = w[0][k] * now[k];
#pragma unroll
                        for (int j = 1; j < W; j++) a += w[j][k] * dp[W - 1 - j][k];
                        o[k] = a + add[k];
                    }
                    if (r >= 0)
                        store_vec<V>(dx + (long long)r * p.C, o);
                    else if (ds0)
                        store_vec<V>(ds0 + (long long)(r + W - 1) * p.C, o);
                }
#pragma unroll
                for (int k = 0; k < V; k++) {
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; j++) dp[j][k] = dp[j + 1][k];
                    dp[W - 2][k] = now[k];
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < V; k++) {
#pragma unroll
        for (int j = 0; j < W; j++) s[threadIdx.y][j][threadIdx.x * V + k] = dw[j][k];
        s[threadIdx.y][W][threadIdx.x * V + k] = db[k];
    }
    __syncthreads();
    for (int i = threadIdx.y * kLanes + threadIdx.x; i < (W + 1) * kLanes * V; i += kLanes * kSub) {
        const int j = i / (kLanes * V), q = i % (kLanes * V);
        const int ch = grp * kLanes * V + q;
        if (ch < p.C) {
            float a = s[0][j][q];
#pragma unroll
            for (int u = 1; u < kSub; u++) a += s[u][j][q];
            p.partial[(((size_t)b * p.pieces + piece) * (W + 1) + j) * p.C + ch] = a;
        }
    }
}

// dweight [C][W] and dbias [C] from the pieces' partials [rows][W + 1][C]: 32 channels and one tap a
// block, 8 threads a sum.  The order of the additions goes by the shape alone.
__global__ void __launch_bounds__(256) ttt_conv_weight_sum_kernel(int rows, int W, int C, const float* __restrict__ partial,
                                                                  float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float s[8][33];
    const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y;
    float a = 0.f;
    if (c < C)
        for (int r = threadIdx.y; r < rows; r += 8) a += partial[((size_t)r * (W + 1) + j) * C + c];
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 8; i++) a += s[i][threadIdx.x];
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
cudaError_t by_width(int W, F f) {
    switch (W) {
        case 2: f(std::integral_constant<int, 2>{}); break;
        case 3: f(std::integral_constant<int, 3>{}); break;
        case 4: f(std::integral_constant<int, 4>{}); break;
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
    p.groups = (a.C + kThreads * v - 1) / (kThreads * v);
    p.ld = a.ld;
    p.x = a.x;
    p.state0 = a.state0;
    p.weight = a.weight;
    p.bias = a.bias;
    p.lengths = a.lengths;
    p.y = a.y;
    p.state_T = a.state_T;
    p.silu = a.silu;
    const long long blocks = (long long)a.B * p.pieces * p.groups;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    return by_width(a.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        if (vec)
            ttt_conv_kernel<T, kV, W><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
        else
            ttt_conv_kernel<T, 1, W><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    });
}

// Tokens a block of the backward takes: 512, halved down to 16 while the launch has fewer threads than
// half of what 148 SMs hold.
int backward_piece(int B, int T, int C, int vec) {
    const long long columns = (long long)B * ((C + kLanes * vec - 1) / (kLanes * vec)) * kLanes * kSub;
    int piece = 512;
    while (piece > 16 && columns * ((T + piece - 1) / piece) < 148LL * 1024) piece /= 2;
    return piece;
}

template <typename T>
cudaError_t backward(const ConvBwdArgs& a, float* workspace, cudaStream_t stream) {
    constexpr int kV = 4;
    const bool vec = a.f.C % kV == 0 && rows_aligned(a.f.x, a.f.ld, kV * sizeof(T), sizeof(T));
    const int v = vec ? kV : 1;
    ConvBwdParams p{};
    p.T = a.f.T;
    p.C = a.f.C;
    p.piece = backward_piece(a.f.B, a.f.T, a.f.C, v);
    p.pieces = a.f.T > 0 ? (a.f.T + p.piece - 1) / p.piece : 1;
    p.groups = (a.f.C + kLanes * v - 1) / (kLanes * v);
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
    p.silu = a.f.silu;
    const long long blocks = (long long)a.f.B * p.pieces * p.groups;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    cudaError_t e = by_width(a.f.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        if (vec)
            ttt_conv_backward_kernel<T, kV, W><<<(unsigned)blocks, dim3(kLanes, kSub), 0, stream>>>(p);
        else
            ttt_conv_backward_kernel<T, 1, W><<<(unsigned)blocks, dim3(kLanes, kSub), 0, stream>>>(p);
    });
    if (e != cudaSuccess) return e;
    ttt_conv_weight_sum_kernel<<<dim3((a.f.C + 31) / 32, a.f.W + 1), dim3(32, 8), 0, stream>>>(
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
    for (int v : {1, 4}) {
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
