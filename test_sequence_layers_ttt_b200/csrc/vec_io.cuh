// Loads and stores of V neighbouring elements of a token row as floats: 16 bytes at once where V
// fills them (the caller has checked the alignment), one element for V = 1.  Rounding to bf16 is to
// nearest, once, at the store.
#pragma once

#include "common.cuh"

namespace ttt {

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;  // elements in 16 bytes
};
template <> struct Elem<float> {
    static constexpr int kVec = 4;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[V]) {
    static_assert(V == 1 || V == 2 || V == 4 || V == 8, "widths in use");
    if constexpr (V == 8) {
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else if constexpr (V == 4) {
        const uint2 r = *reinterpret_cast<const uint2*>(p);
        v[0] = __uint_as_float(r.x << 16);
        v[1] = __uint_as_float(r.x & 0xffff0000u);
        v[2] = __uint_as_float(r.y << 16);
        v[3] = __uint_as_float(r.y & 0xffff0000u);
    } else if constexpr (V == 2) {
        const uint32_t r = *reinterpret_cast<const uint32_t*>(p);
        v[0] = __uint_as_float(r << 16);
        v[1] = __uint_as_float(r & 0xffff0000u);
    } else {
        v[0] = __bfloat162float(*p);
    }
}

template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[V]) {
    static_assert(V == 1 || V == 2 || V == 4 || V == 8, "widths in use");
    if constexpr (V == 1) {
        v[0] = *p;
    } else if constexpr (V == 2) {
        const float2 r = *reinterpret_cast<const float2*>(p);
        v[0] = r.x;
        v[1] = r.y;
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; i++) {
            const float4 r = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = r.x;
            v[4 * i + 1] = r.y;
            v[4 * i + 2] = r.z;
            v[4 * i + 3] = r.w;
        }
    }
}

template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[V]) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint32_t*>(p) = pack_bf16(v[0], v[1]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}

template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = v[0];
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; i++)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
}

// Two floats in one 64-bit register pair, for the packed fp32 instructions of sm_100.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A row's V elements as they come from memory, to be unpacked when they are used
template <typename T, int V>
struct Raw {
    static constexpr int kWords = V * (int)sizeof(T) / 4;  // 0: one bf16
    uint32_t w[kWords > 0 ? kWords : 1];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kWords == 0) {
            w[0] = *reinterpret_cast<const unsigned short*>(p);
        } else if constexpr (kWords == 1) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (kWords == 2) {
            const uint2 r = *reinterpret_cast<const uint2*>(p);
            w[0] = r.x;
            w[1] = r.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 r = reinterpret_cast<const uint4*>(p)[i / 4];
                w[i] = r.x;
                w[i + 1] = r.y;
                w[i + 2] = r.z;
                w[i + 3] = r.w;
            }
        }
    }
    // elements [at, at + V) of a row of `width`: those before 0 or past the end are zeros and are not read
    __device__ __forceinline__ void load_within(const T* row, int at, int width) {
        if (at >= 0 && at + V <= width) {
            load(row + at);
            return;
        }
#pragma unroll
        for (int i = 0; i < (kWords > 0 ? kWords : 1); i++) w[i] = 0u;
        if (at + V <= 0 || at >= width) return;
#pragma unroll
        for (int i = 0; i < V; i++) {
            if (at + i < 0 || at + i >= width) continue;
            if constexpr (sizeof(T) == 4)
                w[i] = reinterpret_cast<const uint32_t*>(row)[at + i];
            else
                w[i / 2] |= (uint32_t) reinterpret_cast<const unsigned short*>(row)[at + i] << (i % 2 * 16);
        }
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = __uint_as_float(w[i]);
        } else if constexpr (V == 1) {
            v[0] = __uint_as_float(w[0] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i++) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

// The same values as pairs (an even V)
template <typename T, int V>
__device__ __forceinline__ void pairs_of(const Raw<T, V>& r, f2 (&o)[V / 2]) {
    float v[V];
    r.get(v);
#pragma unroll
    for (int i = 0; i < V / 2; i++) o[i] = pack2(v[2 * i], v[2 * i + 1]);
}

// Elements [at, at + V) of a row of `width` that lie in it
template <int V, typename T>
__device__ __forceinline__ void store_within(T* row, int at, int width, const float (&v)[V]) {
    if (at >= 0 && at + V <= width) {
        store_vec<V>(row + at, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; i++)
        if (at + i >= 0 && at + i < width) {
            const float one[1] = {v[i]};
            store_vec<1>(row + at + i, one);
        }
}

// 2^x and 1 / x by the special-function unit, tiny results flushed to zero (the forms that keep them cost
// four instructions more)
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// V neighbouring values as pairs (V = 1: one pair with a zero)
template <int V>
__device__ __forceinline__ void to_pairs(const float (&v)[V], f2 (&o)[(V + 1) / 2]) {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; i++) o[i] = pack2(v[2 * i], 2 * i + 1 < V ? v[(2 * i + 1) % V] : 0.f);
}
template <int V>
__device__ __forceinline__ void from_pairs(const f2 (&o)[(V + 1) / 2], float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; i++) {
        float lo, hi;
        unpack2(o[i], lo, hi);
        v[2 * i] = lo;
        if (2 * i + 1 < V) v[(2 * i + 1) % V] = hi;
    }
}

// logistic function 1 / (1 + e^-x); at the ends e^-x is 0 or infinity and the result 1 or 0
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-1.4426950408889634f * x)); }

__device__ __forceinline__ f2 sigmoid2(f2 x) {
    float lo, hi;
    unpack2(mul2(x, pack2(-1.4426950408889634f, -1.4426950408889634f)), lo, hi);
    unpack2(add2(pack2(ex2(lo), ex2(hi)), pack2(1.f, 1.f)), lo, hi);
    return pack2(rcp(lo), rcp(hi));
}

}  // namespace ttt
