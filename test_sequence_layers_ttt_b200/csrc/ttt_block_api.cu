// Host layer of the operators around the sequence layer (include/ttt.h, second half): argument checks
// and launches.  Checks run on the host alone; a call that fails one launches nothing.
#include <cfloat>
#include <climits>

#include "api_util.h"

namespace {

using namespace ttt;

size_t size_of(ttt_dtype t) { return t == TTT_BF16 ? 2 : 4; }
bool known(ttt_dtype t) { return t == TTT_BF16 || t == TTT_F32; }
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Bytes that `rows` rows of `width` elements, `ld` apart, span
size_t span_of(size_t rows, size_t width, long long ld, size_t es) {
    return rows == 0 ? 0 : ((rows - 1) * (size_t)ld + width) * es;
}

template <size_t n>
bool any_null(const void* const (&p)[n]) {
    for (const void* q : p)
        if (!q) return true;
    return false;
}
template <size_t n>
bool any_unaligned(const void* const (&p)[n]) {
    for (const void* q : p)
        if (q && !aligned16(q)) return true;
    return false;
}

// No output overlaps an input or another output; an output may be exactly the one input that allowed[o]
// names (-1: none).
template <size_t no, size_t ni>
ttt_status no_overlap(const Span (&outs)[no], const int (&allowed)[no], const Span (&ins)[ni]) {
    return check_aliasing(outs, (int)no, ins, allowed, (int)ni);
}

// Token numbers, and those of the tile that one falls in, stay below 2^31
bool tokens_fit(int B, int T) { return (long long)B * T < (1LL << 31) - (1LL << 16); }

ttt_status launched(cudaError_t e, ttt_stream_t stream) { return finish(e, reinterpret_cast<cudaStream_t>(stream)); }

// ---------------------------------------------------------------- norm
ttt_status check_norm_shape(int B, int T, int d, ttt_dtype dtype, float eps) {
    if (B < 1 || T < 1 || d < 1 || !tokens_fit(B, T)) return TTT_ERR_SHAPE;
    if (!(eps > 0.f)) return TTT_ERR_SHAPE;
    if (!known(dtype)) return TTT_ERR_DTYPE;
    if (d > kNormMaxWidth) return TTT_ERR_UNSUPPORTED;
    return TTT_OK;
}

// A row is read whole before it is written, so an output may be exactly x or residual.
ttt_status check_norm(const NormArgs& a, bool q8) {
    ttt_status st = check_norm_shape(a.B, a.T, a.d, a.dtype, a.eps);
    if (st != TTT_OK) return st;
    if (any_null({a.x, a.weight, a.y}) || (q8 && !a.scale)) return TTT_ERR_NULL;
    if (any_unaligned({a.x, a.residual, a.weight, a.y, a.h, a.scale})) return TTT_ERR_ALIGN;
    const size_t n = (size_t)a.B * a.T * a.d, bytes = n * size_of(a.dtype);
    const Span x{a.x, bytes}, r{a.residual, a.residual ? bytes : 0}, w{a.weight, (size_t)a.d * 4};
    const Span y{a.y, q8 ? n : bytes}, h{a.h, a.h ? bytes : 0}, s{a.scale, q8 ? (size_t)a.B * a.T * 4 : 0};
    for (const Span& o : {y, h, s}) {
        if (overlap(o, w)) return TTT_ERR_ALIAS;
        for (const Span& i : {x, r}) {
            const bool same = o.p == i.p && o.bytes == i.bytes && o.p != a.scale;
            if (overlap(o, i) && !same) return TTT_ERR_ALIAS;
        }
    }
    if (overlap(y, h) || overlap(y, s) || overlap(h, s)) return TTT_ERR_ALIAS;
    return TTT_OK;
}

ttt_status check_norm_backward(const NormBwdArgs& a, const void* workspace, size_t workspace_bytes, size_t need) {
    ttt_status st = check_norm_shape(a.B, a.T, a.d, a.dtype, a.eps);
    if (st != TTT_OK) return st;
    if (any_null({a.h, a.weight, a.dy, a.dh, a.dweight})) return TTT_ERR_NULL;
    if (any_unaligned({a.h, a.weight, a.dy, a.dh_in, a.dh, a.dweight, workspace})) return TTT_ERR_ALIGN;
    if (!workspace || workspace_bytes < need) return TTT_ERR_WORKSPACE;
    const size_t bytes = (size_t)a.B * a.T * a.d * size_of(a.dtype), w = (size_t)a.d * 4;
    const Span ins[] = {{a.dy, bytes}, {a.dh_in, a.dh_in ? bytes : 0}, {a.h, bytes}, {a.weight, w}, {workspace, need}};
    const Span outs[] = {{a.dh, bytes}, {a.dweight, w}};
    const int allowed[] = {a.dh == a.dy ? 0 : 1, -1};
    return no_overlap(outs, allowed, ins);
}

// ---------------------------------------------------------------- 8-bit prologue
ttt_status check_prologue_q8(const PrologueArgs& a, const PrologueScales& s) {
    if (a.B < 1 || a.T < 1 || a.H < 1 || a.d_model < 1 || !tokens_fit(a.B, a.T)) return TTT_ERR_SHAPE;
    if (!(a.rope_base > 1.f && a.rope_base <= FLT_MAX) || !(a.eta_base == a.eta_base)) return TTT_ERR_SHAPE;
    if (!prologue_q8_supports(a.B, a.T, a.H, a.d, a.d_model)) return TTT_ERR_UNSUPPORTED;
    const void* const req[] = {a.x, s.x, a.theta_q, s.q, a.theta_k, s.k, a.theta_v, s.v, a.theta_lr, s.lr,
                               a.b_lr, a.Q, a.K, a.V, a.eta};
    if (any_null(req)) return TTT_ERR_NULL;
    if (any_unaligned(req)) return TTT_ERR_ALIGN;
    const size_t tok = (size_t)a.B * a.T, hd = (size_t)a.H * a.d, w = (size_t)a.d_model * hd, h4 = (size_t)a.H * 4;
    const Span ins[] = {{a.x, tok * a.d_model}, {s.x, tok * 4}, {a.theta_q, w}, {s.q, hd * 4}, {a.theta_k, w},
                        {s.k, hd * 4}, {a.theta_v, w}, {s.v, hd * 4}, {a.theta_lr, (size_t)a.H * a.d_model},
                        {s.lr, h4}, {a.b_lr, h4}};
    const Span outs[] = {{a.Q, tok * hd * 2}, {a.K, tok * hd * 2}, {a.V, tok * hd * 2}, {a.eta, tok * h4}};
    const int allowed[] = {-1, -1, -1, -1};
    return no_overlap(outs, allowed, ins);
}

// ---------------------------------------------------------------- convolution
// The inputs' checks; `ins` receives their spans.
ttt_status check_conv_inputs(const ConvArgs& a, Span (&ins)[5]) {
    if (a.B < 1 || a.T < 0 || a.C < 1 || !tokens_fit(a.B, a.T) || a.ld < a.C) return TTT_ERR_SHAPE;
    if (!known(a.dtype)) return TTT_ERR_DTYPE;
    if (a.W < 2 || a.W > kConvMaxWidth) return TTT_ERR_UNSUPPORTED;
    if (!a.weight || (a.T > 0 && !a.x)) return TTT_ERR_NULL;
    const size_t es = size_of(a.dtype), C = a.C;
    if (!aligned_to(a.x, es) || any_unaligned({a.weight, a.bias, a.state0, a.lengths})) return TTT_ERR_ALIGN;
    ins[0] = {a.state0, a.state0 ? (size_t)a.B * (a.W - 1) * C * es : 0};
    ins[1] = {a.x, span_of((size_t)a.B * a.T, C, a.ld, es)};
    ins[2] = {a.weight, C * a.W * 4};
    ins[3] = {a.bias, a.bias ? C * 4 : 0};
    ins[4] = {a.lengths, a.lengths ? (size_t)a.B * 4 : 0};
    return TTT_OK;
}

ttt_status check_conv(const ConvArgs& a) {
    Span ins[5];
    ttt_status st = check_conv_inputs(a, ins);
    if (st != TTT_OK) return st;
    if (a.T > 0 && !a.y) return TTT_ERR_NULL;
    if (any_unaligned({a.y, a.state_T})) return TTT_ERR_ALIGN;
    const size_t es = size_of(a.dtype);
    const Span outs[] = {{a.y, (size_t)a.B * a.T * a.C * es},
                         {a.state_T, a.state_T ? (size_t)a.B * (a.W - 1) * a.C * es : 0}};
    const int allowed[] = {-1, 0};
    return no_overlap(outs, allowed, ins);
}

ttt_status check_conv_backward(const ConvBwdArgs& a, const void* workspace, size_t workspace_bytes, size_t need) {
    Span in[5];
    const ConvArgs& f = a.f;
    ttt_status st = check_conv_inputs(f, in);
    if (st != TTT_OK) return st;
    if (!a.dweight || (f.T > 0 && (!a.dy || !a.dx))) return TTT_ERR_NULL;
    if (any_unaligned({a.dy, a.dstate_T, a.dx, a.dweight, a.dbias, a.dstate0, workspace})) return TTT_ERR_ALIGN;
    if (!workspace || workspace_bytes < need) return TTT_ERR_WORKSPACE;
    const size_t es = size_of(f.dtype), rows = (size_t)f.B * f.T * f.C * es, st_b = (size_t)f.B * (f.W - 1) * f.C * es;
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], {a.dy, rows}, {a.dstate_T, a.dstate_T ? st_b : 0},
                        {workspace, need}};
    const Span outs[] = {{a.dx, rows}, {a.dweight, (size_t)f.C * f.W * 4}, {a.dbias, a.dbias ? (size_t)f.C * 4 : 0},
                         {a.dstate0, a.dstate0 ? st_b : 0}};
    const int allowed[] = {-1, -1, -1, -1};
    return no_overlap(outs, allowed, ins);
}

// ---------------------------------------------------------------- selective scan
ttt_status check_ssm_inputs(const SsmArgs& a, Span (&ins)[10]) {
    if (a.B < 1 || a.T < 0 || a.C < 1 || a.N < 1 || !tokens_fit(a.B, a.T)) return TTT_ERR_SHAPE;
    if (a.ld_u < a.C || a.ld_dt < a.C || a.ld_b < a.N || a.ld_c < a.N || (a.z && a.ld_z < a.C)) return TTT_ERR_SHAPE;
    if (!known(a.dtype)) return TTT_ERR_DTYPE;
    if (a.N > kSsmMaxStates) return TTT_ERR_UNSUPPORTED;
    if (!a.A || (a.T > 0 && (!a.u || !a.dt || !a.Bm || !a.Cm))) return TTT_ERR_NULL;
    const size_t es = size_of(a.dtype), C = a.C, rows = (size_t)a.B * a.T;
    for (const void* p : {a.u, a.dt, a.Bm, a.Cm, a.z})
        if (!aligned_to(p, es)) return TTT_ERR_ALIGN;
    if (any_unaligned({a.dt_bias, a.A, a.D, a.h0, a.lengths})) return TTT_ERR_ALIGN;
    ins[0] = {a.h0, a.h0 ? (size_t)a.B * C * a.N * 4 : 0};
    ins[1] = {a.u, span_of(rows, C, a.ld_u, es)};
    ins[2] = {a.dt, span_of(rows, C, a.ld_dt, es)};
    ins[3] = {a.Bm, span_of(rows, a.N, a.ld_b, es)};
    ins[4] = {a.Cm, span_of(rows, a.N, a.ld_c, es)};
    ins[5] = {a.z, a.z ? span_of(rows, C, a.ld_z, es) : 0};
    ins[6] = {a.dt_bias, a.dt_bias ? C * 4 : 0};
    ins[7] = {a.A, C * a.N * 4};
    ins[8] = {a.D, a.D ? C * 4 : 0};
    ins[9] = {a.lengths, a.lengths ? (size_t)a.B * 4 : 0};
    return TTT_OK;
}

ttt_status check_ssm(const SsmArgs& a) {
    Span ins[10];
    ttt_status st = check_ssm_inputs(a, ins);
    if (st != TTT_OK) return st;
    if (!a.h_T || (a.T > 0 && !a.y)) return TTT_ERR_NULL;
    if (any_unaligned({a.y, a.h_T})) return TTT_ERR_ALIGN;
    const Span outs[] = {{a.y, (size_t)a.B * a.T * a.C * size_of(a.dtype)}, {a.h_T, (size_t)a.B * a.C * a.N * 4}};
    const int allowed[] = {-1, 0};
    return no_overlap(outs, allowed, ins);
}

ttt_status check_ssm_backward(const SsmBwdArgs& a, const void* workspace, size_t workspace_bytes, size_t need) {
    Span in[10];
    const SsmArgs& f = a.f;
    ttt_status st = check_ssm_inputs(f, in);
    if (st != TTT_OK) return st;
    if (!a.dA || (f.T > 0 && (!a.dy || !a.du || !a.ddt || !a.dB || !a.dC || (f.z && !a.dz)))) return TTT_ERR_NULL;
    if (a.dz && !f.z) return TTT_ERR_NULL;
    if (any_unaligned({a.dy, a.dh_T, a.du, a.ddt, a.dz, a.dA, a.dB, a.dC, a.dD, a.ddt_bias, a.dh0, workspace}))
        return TTT_ERR_ALIGN;
    if (!workspace || workspace_bytes < need) return TTT_ERR_WORKSPACE;
    const size_t C = f.C, N = f.N, tok = (size_t)f.B * f.T, rows = tok * C * size_of(f.dtype), bc = tok * N * 4;
    const size_t hb = (size_t)f.B * C * N * 4;
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7], in[8], in[9],
                        {a.dy, rows}, {a.dh_T, a.dh_T ? hb : 0}, {workspace, need}};
    const Span outs[] = {{a.du, rows}, {a.ddt, rows}, {a.dz, a.dz ? rows : 0}, {a.dA, C * N * 4}, {a.dB, bc}, {a.dC, bc},
                         {a.dD, a.dD ? C * 4 : 0}, {a.ddt_bias, a.ddt_bias ? C * 4 : 0}, {a.dh0, a.dh0 ? hb : 0}};
    const int allowed[] = {-1, -1, -1, -1, -1, -1, -1, -1, -1};
    return no_overlap(outs, allowed, ins);
}

}  // namespace

extern "C" {

ttt_status ttt_rmsnorm_forward(int B, int T, int d, ttt_dtype dtype, float eps, const void* x, const void* residual,
                               const float* weight, void* y, void* h, ttt_stream_t stream) {
    const NormArgs a{B, T, d, dtype, eps, x, residual, weight, y, h, nullptr};
    const ttt_status st = check_norm(a, false);
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_rmsnorm(a, reinterpret_cast<cudaStream_t>(stream)), stream);
}

ttt_status ttt_rmsnorm_q8_forward(int B, int T, int d, ttt_dtype dtype, float eps, const void* x,
                                  const void* residual, const float* weight, void* q, float* scale, void* h,
                                  ttt_stream_t stream) {
    const NormArgs a{B, T, d, dtype, eps, x, residual, weight, q, h, scale};
    const ttt_status st = check_norm(a, true);
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_rmsnorm(a, reinterpret_cast<cudaStream_t>(stream)), stream);
}

size_t ttt_rmsnorm_backward_workspace_size(int B, int T, int d, ttt_dtype dtype) {
    return rmsnorm_backward_workspace_bytes(B, T, d, dtype);
}

ttt_status ttt_rmsnorm_backward(int B, int T, int d, ttt_dtype dtype, float eps, const void* h, const float* weight,
                                const void* dy, const void* dh_in, void* dh, float* dweight, void* workspace,
                                size_t workspace_bytes, ttt_stream_t stream) {
    const NormBwdArgs a{B, T, d, dtype, eps, h, weight, dy, dh_in, dh, dweight};
    const ttt_status st =
        check_norm_backward(a, workspace, workspace_bytes, rmsnorm_backward_workspace_bytes(B, T, d, dtype));
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_rmsnorm_backward(a, static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream)),
                    stream);
}

ttt_status ttt_prologue_q8_forward(int B, int T, int H, int d, int d_model, int pos0, float eta_base, float rope_base,
                                   int rotary, const void* x, const float* scale_x, const void* theta_q,
                                   const float* scale_q, const void* theta_k, const float* scale_k,
                                   const void* theta_v, const float* scale_v, const void* theta_lr,
                                   const float* scale_lr, const float* b_lr, void* Q, void* K, void* V, float* eta,
                                   ttt_stream_t stream) {
    const PrologueArgs a{B, T, H, d, d_model, pos0, rotary ? 1 : 0, eta_base, rope_base, x, theta_q, theta_k,
                         theta_v, theta_lr, b_lr, Q, K, V, eta};
    const PrologueScales s{scale_x, scale_q, scale_k, scale_v, scale_lr};
    const ttt_status st = check_prologue_q8(a, s);
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_prologue_q8(a, s, reinterpret_cast<cudaStream_t>(stream)), stream);
}

ttt_status ttt_conv_forward(int B, int T, int C, int width, ttt_dtype dtype, int silu, long long ld_x, const void* x,
                            const float* weight, const float* bias, const void* state0, const int* lengths, void* y,
                            void* state_T, ttt_stream_t stream) {
    const ConvArgs a{B, T, C, width, dtype, silu, ld_x, x, weight, bias, state0, lengths, y, state_T};
    const ttt_status st = check_conv(a);
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_conv(a, reinterpret_cast<cudaStream_t>(stream)), stream);
}

ttt_status ttt_conv_decode(int B, int T, int C, int width, ttt_dtype dtype, int silu, long long ld_x, const void* x,
                           const float* weight, const float* bias, void* state, void* y, ttt_stream_t stream) {
    if (!state) return TTT_ERR_NULL;
    return ttt_conv_forward(B, T, C, width, dtype, silu, ld_x, x, weight, bias, state, nullptr, y, state, stream);
}

size_t ttt_conv_backward_workspace_size(int B, int T, int C, int width) {
    return conv_backward_workspace_bytes(B, T, C, width);
}

ttt_status ttt_conv_backward(int B, int T, int C, int width, ttt_dtype dtype, int silu, long long ld_x, const void* x,
                             const float* weight, const float* bias, const void* state0, const int* lengths,
                             const void* dy, const void* dstate_T, void* dx, float* dweight, float* dbias,
                             void* dstate0, void* workspace, size_t workspace_bytes, ttt_stream_t stream) {
    const ConvBwdArgs a{{B, T, C, width, dtype, silu, ld_x, x, weight, bias, state0, lengths, nullptr, nullptr},
                        dy, dstate_T, dx, dweight, dbias, dstate0};
    const ttt_status st =
        check_conv_backward(a, workspace, workspace_bytes, conv_backward_workspace_bytes(B, T, C, width));
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_conv_backward(a, static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream)),
                    stream);
}

ttt_status ttt_ssm_forward(int B, int T, int C, int N, ttt_dtype dtype, int dt_softplus, long long ld_u,
                           long long ld_dt, long long ld_b, long long ld_c, long long ld_z, const void* u,
                           const void* dt, const float* dt_bias, const float* A, const void* Bm, const void* Cm,
                           const float* D, const void* z, const float* h0, const int* lengths, void* y, float* h_T,
                           ttt_stream_t stream) {
    const SsmArgs a{B, T, C, N, dtype, dt_softplus, ld_u, ld_dt, ld_b, ld_c, ld_z, u, dt, dt_bias, A, Bm, Cm, D, z,
                    h0, lengths, y, h_T};
    const ttt_status st = check_ssm(a);
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_ssm_forward(a, reinterpret_cast<cudaStream_t>(stream)), stream);
}

ttt_status ttt_ssm_decode(int B, int T, int C, int N, ttt_dtype dtype, int dt_softplus, long long ld_u,
                          long long ld_dt, long long ld_b, long long ld_c, long long ld_z, const void* u,
                          const void* dt, const float* dt_bias, const float* A, const void* Bm, const void* Cm,
                          const float* D, const void* z, float* h, void* y, ttt_stream_t stream) {
    const SsmArgs a{B, T, C, N, dtype, dt_softplus, ld_u, ld_dt, ld_b, ld_c, ld_z, u, dt, dt_bias, A, Bm, Cm, D, z,
                    h, nullptr, y, h};
    const ttt_status st = check_ssm(a);
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_ssm_token(a, reinterpret_cast<cudaStream_t>(stream)), stream);
}

size_t ttt_ssm_backward_workspace_size(int B, int T, int C, int N) { return ssm_backward_workspace_bytes(B, T, C, N); }

ttt_status ttt_ssm_backward(int B, int T, int C, int N, ttt_dtype dtype, int dt_softplus, long long ld_u,
                            long long ld_dt, long long ld_b, long long ld_c, long long ld_z, const void* u,
                            const void* dt, const float* dt_bias, const float* A, const void* Bm, const void* Cm,
                            const float* D, const void* z, const float* h0, const int* lengths, const void* dy,
                            const float* dh_T, void* du, void* ddt, float* dA, float* dB, float* dC, float* dD,
                            void* dz, float* ddt_bias, float* dh0, void* workspace, size_t workspace_bytes,
                            ttt_stream_t stream) {
    const SsmBwdArgs a{{B, T, C, N, dtype, dt_softplus, ld_u, ld_dt, ld_b, ld_c, ld_z, u, dt, dt_bias, A, Bm, Cm, D, z,
                        h0, lengths, nullptr, nullptr},
                       dy, dh_T, du, ddt, dz, dA, dB, dC, dD, ddt_bias, dh0};
    const ttt_status st = check_ssm_backward(a, workspace, workspace_bytes, ssm_backward_workspace_bytes(B, T, C, N));
    if (st != TTT_OK) return st;
    if (!prepare()) return TTT_ERR_CUDA;
    return launched(launch_ssm_backward(a, static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream)), stream);
}

}  // extern "C"
