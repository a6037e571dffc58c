// Arithmetic of the selective scan shared by its forward, decode and backward kernels.
//
// The decay a = e^(dt A) = 2^x with x = dt A log2(e).  Where a is close to 1 the state remembers about
// 1 / |x| tokens, so an error of a that does not average out grows by that factor; the special-function
// unit's 2^x is off by up to 2^-22 and, between -1/16 and 0, by 2.5e-8 low on average (measured over
// 2^20 points an octave).  So for |x| < 1/16 the decay is 1 + x q(x) with q the quadratic that fits
// (2^x - 1) / x on [-1/16, 0] to 1.3e-7 (Remez exchange), or, where x may be positive, the cubic that fits it
// on [-1/16, 1/16] to 1e-8 (interpolation at the zeros of a Chebyshev polynomial; the quadratic is off by 1e-5
// at +1/16): 1 - a is then right to 1.3e-7 whatever its size, and only the last rounding, which is to
// nearest, is left.  Beyond it the unit's result stands: its error counts at most 16 times there.
// The cost is three or four of the pipe's fused multiply-adds a state beside one special-function result
// (16 a clock an SM), which stays the bound.  With the cubic for all states the scan of many channels took 1456 us
// against 1414 (1.3B width, 32k tokens), so there, and in the gradient's first pass, a warp asks once whether any of its
// states grows; elsewhere it is used for all (gradient of 8 x 2048 x 1536: 1.02 ms against 1.00).
#pragma once

#include "vec_io.cuh"

namespace ttt {
namespace ssm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSmall = 0.0625f;
constexpr float kQ0 = 0x1.62e42ep-1f, kQ1 = 0x1.ebf0e6p-3f, kQ2 = 0x1.bf5dd8p-5f;                              // x <= 0
constexpr float kG0 = 0x1.62e430p-1f, kG1 = 0x1.ebfbe0p-3f, kG2 = 0x1.c6bb7ap-5f, kG3 = 0x1.3b2fc4p-7f;  // any x

// A log2(e), infinity as the largest float: a step of zero, as padding has it, then still leaves the state as it is
__device__ __forceinline__ float rate(float A) {
    const float v = A * kLog2e;
    return fabsf(v) == INFINITY ? copysignf(3.4028235e38f, v) : v;
}

__device__ __forceinline__ float decay(float x) {
    const float q = fmaf(fmaf(fmaf(kG3, x, kG2), x, kG1), x, kG0);
    const float near_one = fmaf(q, x, 1.f);
    return fabsf(x) < kSmall ? near_one : ex2(x);
}

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1]: log(1 + e) = 2 atanh(s), s = e / (2 + e) in
// (0, 1/3], by an even polynomial that fits 2 atanh(s) / s to 8e-9; right to a few 1e-7 of the result for x > -5.  Below,
// where the result is e^x, the rounding of x log2(e) counts about |x| 2^-24 of it (2e-6 at -40); below -87 it is 0.
__device__ __forceinline__ float softplus(float x) {
    const float e = ex2(-kLog2e * fabsf(x));
    const float s = e * rcp(2.f + e), w = s * s;
    float p = 0x1.208bd0p-2f;
    p = fmaf(p, w, 0x1.1e510ap-2f);
    p = fmaf(p, w, 0x1.99dae6p-2f);
    p = fmaf(p, w, 0x1.5554e0p-1f);
    p = fmaf(p, w, 2.f);
    return fmaf(s, p, fmaxf(x, 0.f));
}

// 2^x in the place of `near_one` where |x| >= 1/16: one comparison and a predicated instruction
__device__ __forceinline__ void ex2_beyond(float& near_one, float x) {
    asm("{\n .reg .pred p;\n .reg .f32 m;\n abs.f32 m, %1;\n setp.ge.f32 p, m, 0f3D800000;\n"
        " @p ex2.approx.ftz.f32 %0, %1;\n}"
        : "+f"(near_one)
        : "f"(x));
}
// Whether any state of the warp may have a positive x
__device__ __forceinline__ bool warp_grows(bool softplus, const float (&a2)[4]) {
    return __any_sync(0xffffffffu, !softplus || fmaxf(fmaxf(a2[0], a2[1]), fmaxf(a2[2], a2[3])) > 0.f);
}

// decay() of 2 kPairs values, x in pairs, all x <= 0 unless kGrow; step by step over all pairs, so that a warp has
// independent work at every step
template <bool kGrow, int kPairs>
__device__ __forceinline__ void decays(float (&a)[2 * kPairs], const f2 (&x)[kPairs]) {
    const auto step = [&](f2(&q)[kPairs], float c) {
        const f2 c2 = pack2(c, c);
#pragma unroll
        for (int i = 0; i < kPairs; i++) q[i] = fma2(q[i], x[i], c2);
    };
    const f2 one = pack2(1.f, 1.f), top = kGrow ? pack2(kG3, kG3) : pack2(kQ2, kQ2);
    f2 q[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; i++) q[i] = top;
    if (kGrow) step(q, kG2);
    step(q, kGrow ? kG1 : kQ1);
    step(q, kGrow ? kG0 : kQ0);
#pragma unroll
    for (int i = 0; i < kPairs; i++) q[i] = fma2(q[i], x[i], one);
#pragma unroll
    for (int i = 0; i < kPairs; i++) {
        float x0, x1;
        unpack2(x[i], x0, x1);
        unpack2(q[i], a[2 * i], a[2 * i + 1]);
        ex2_beyond(a[2 * i], x0);
        ex2_beyond(a[2 * i + 1], x1);
    }
}

// v carried over many tokens, v a + e.  A growing state's a may pass the largest float where v a does not, so it comes
// as two factors of about its root; where they overflow too, a v of zero still becomes e.
__device__ __forceinline__ float carried(float v, float a0, float a1, float e) { return v == 0.f ? e : fmaf(a0 * v, a1, e); }

__device__ __forceinline__ int length_of(const int* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

}  // namespace ssm
}  // namespace ttt
