// channel.cuh -- shared pieces of the channel operators (RMS norm, linear
// layer, gated projections): tensors seen as rows (pixels or tokens) by
// channels, activations with their derivatives, and typed loads and stores.
//
// Whatever a kernel reads, the grid ahead of it may still be writing when it starts (a
// norm's row scales, an output that is the next layer's bias): it is read after
// griddep_wait and by plain loads, never by the read-only path, whose data must not
// change while the kernel runs and whose loads may be moved above the wait.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <type_traits>

#include "internal.h"

namespace dlc {

// Element offset of row m's channel 0 (channel c is c * cs further).
__device__ __forceinline__ long long row_off(const RowMap &r, long long m) {
    if (r.uniform) return m * r.ld;
    const long long n = m / r.hw;
    const int rem = (int)(m - n * r.hw);
    const int h = rem / r.w;
    return n * r.s0 + h * r.s2 + (long long)(rem - h * r.w) * r.s3;
}

__device__ __forceinline__ float bf16_bits_f32(uint32_t b) { return __uint_as_float(b << 16); }

// Two FP32 values rounded to nearest even into one word of BF16 (a in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// What rounding to BF16 leaves of v (nothing of an infinity).
__device__ __forceinline__ float bf16_rest(float v) {
    const float r = bf16_bits_f32(pack_bf16(v, 0.f) & 0xffffu);
    return isinf(r) ? 0.f : v - r;
}

// Two FP32 values rounded to nearest even into E4M3, saturating at +-448 (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// One element of a FLOAT, BFLOAT16 or FLOAT8_E4M3 array as FP32, and back.
__device__ __forceinline__ float load_elem(const void *p, int dt, long long i) {
    if (dt == DLC_DATA_FLOAT) return static_cast<const float *>(p)[i];
    if (dt == DLC_DATA_BFLOAT16) return bf16_bits_f32(static_cast<const unsigned short *>(p)[i]);
    __nv_fp8_e4m3 v;
    v.__x = static_cast<const unsigned char *>(p)[i];
    return float(v);
}

// n elements `stride` apart, FLOAT or BFLOAT16, as FP32; element i only where
// in(i), zero elsewhere.  The storage type is looked at once, outside, so that
// the loads are in flight together (a load behind its own branch is waited for
// before the next one starts).
template <int N, typename In>
__device__ __forceinline__ void load_elems(const void *p, int dt, long long off, long long stride, In in, float *v) {
    if (dt == DLC_DATA_BFLOAT16) {
        const unsigned short *s = static_cast<const unsigned short *>(p) + off;
        unsigned short w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = in(i) ? s[i * stride] : (unsigned short)0;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = bf16_bits_f32(w[i]);
    } else {
        const float *s = static_cast<const float *>(p) + off;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = in(i) ? s[i * stride] : 0.f;
    }
}

__device__ __forceinline__ void store_elem(void *p, int dt, long long i, float v) {
    if (dt == DLC_DATA_FLOAT)
        static_cast<float *>(p)[i] = v;
    else if (dt == DLC_DATA_BFLOAT16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<unsigned char *>(p)[i] = (unsigned char)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// Four consecutive channels n .. n+3 of a row, `cols` of which exist; `vec`:
// the tensor takes four-element accesses (dlc_vec4_rows).
__device__ __forceinline__ void load4(const RowTensor &t, long long off, int n, int cols, bool vec,
                                      float (&v)[4]) {
    if (vec && cols >= 4) {
        if (t.dt == DLC_DATA_BFLOAT16) {
            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const unsigned short *>(t.p) + off + n);
            v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
            v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(t.p) + off + n);
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        }
    } else {
        load_elems<4>(t.p, t.dt, off + (long long)n * t.m.cs, t.m.cs, [&](int i) { return i < cols; }, v);
    }
}

__device__ __forceinline__ void store4(const RowTensor &t, long long off, long long n, int cols, bool vec,
                                           const float (&v)[4]) {
    if (vec && cols >= 4) {
        if (t.dt == DLC_DATA_BFLOAT16)
            *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(t.p) + off + n) =
                make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(t.p) + off + n) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < cols) store_elem(t.p, t.dt, off + (n + i) * t.m.cs, v[i]);
    }
}

// Two FP32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)), "l"(*reinterpret_cast<const unsigned long long *>(&b)),
          "l"(*reinterpret_cast<const unsigned long long *>(&c)));
    return *reinterpret_cast<const float2 *>(&d);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)), "l"(*reinterpret_cast<const unsigned long long *>(&b)));
    return *reinterpret_cast<const float2 *>(&d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)), "l"(*reinterpret_cast<const unsigned long long *>(&b)));
    return *reinterpret_cast<const float2 *>(&d);
}

// The two BF16 values of a word.
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 2^v and 1 / v by the special-function unit (a few units in the last place of
// FP32; results below the normal range are zero).
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float recip_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Pair i of an array.
__device__ __forceinline__ float2 get2(const float *v, int i) { return make_float2(v[2 * i], v[2 * i + 1]); }
__device__ __forceinline__ void set2(float *v, int i, float2 w) { v[2 * i] = w.x, v[2 * i + 1] = w.y; }

__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }

// Phi(v), the standard normal distribution function, from e = exp(-v^2 / 2):
// Phi(-|v|) = e t (a1 + a2 t + ... + a8 t^7), t = 1 / (1 + 0.305 |v|).  The a were fitted
// to the smallest largest relative error over 0 <= |v| <= 14.5 (a linear program on 4000
// points; e leaves FP32 behind 13.2): 1e-7, so the tail keeps its digits as
// erff's 1 + erf does not; the density shares the exponential.
__device__ __forceinline__ float2 gelu_phi(float2 v, float2 e) {
    const float2 d = fma2(make_float2(fabsf(v.x), fabsf(v.y)), pair_of(0.305f), pair_of(1.f));
    const float2 t = make_float2(recip_fast(d.x), recip_fast(d.y));
    float2 q = fma2(t, pair_of(0.0366388683f), pair_of(-0.1527461f));
    q = fma2(q, t, pair_of(0.185314941f));
    q = fma2(q, t, pair_of(-0.0376206951f));
    q = fma2(q, t, pair_of(0.120840406f));
    q = fma2(q, t, pair_of(0.10347369f));
    q = fma2(q, t, pair_of(0.122458682f));
    q = fma2(q, t, pair_of(0.121640242f));
    q = mul2(q, mul2(t, e));
    const float2 c = fma2(q, pair_of(-1.f), pair_of(1.f));
    return make_float2(v.x < 0.f ? q.x : c.x, v.y < 0.f ? q.y : c.y);
}

// 1 / (1 + exp(-v)), exp(-v^2 / 2)
__device__ __forceinline__ float2 logistic(float2 v) {
    const float2 a = mul2(v, pair_of(-1.4426950408889634f));
    const float2 d = add2(make_float2(exp2_fast(a.x), exp2_fast(a.y)), pair_of(1.f));
    return make_float2(recip_fast(d.x), recip_fast(d.y));
}

__device__ __forceinline__ float2 gauss(float2 v) {
    const float2 a = mul2(mul2(v, v), pair_of(-0.5f * 1.4426950408889634f));
    return make_float2(exp2_fast(a.x), exp2_fast(a.y));
}

// f(v) of the linear and gated epilogues, two values at a time: the epilogue's
// instructions bound the products of a short reduction (GELU of a 256 x 256 tile
// cost 3.6 us one value at a time, 2.6 us this way, 0.35 of them for the precision of its
// tail).  Relative errors, down to where FP32's normal range ends: GELU 4e-6 + 1e-7 v^2, SILU and sigmoid 1e-6 + 2e-7 |v| (the exponent's
// rounding grows with it).  SILU and GELU of -inf are -inf * 0 = NaN, as their formulas say.
template <int ACT>
__device__ __forceinline__ float2 act_f2(float2 v) {
    if constexpr (ACT == DLC_ACTIVATION_RELU) return make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);  // NaN stays NaN
    if constexpr (ACT == DLC_ACTIVATION_SIGMOID) return logistic(v);
    if constexpr (ACT == DLC_ACTIVATION_TANH) return make_float2(tanhf(v.x), tanhf(v.y));
    if constexpr (ACT == DLC_ACTIVATION_SILU) return mul2(v, logistic(v));
    if constexpr (ACT == DLC_ACTIVATION_GELU) return mul2(v, gelu_phi(v, gauss(v)));
    return v;
}

template <int ACT>
__device__ __forceinline__ float act_f(float v) { return act_f2<ACT>(pair_of(v)).x; }

// f(v) and f'(v).
template <int ACT>
__device__ __forceinline__ void act_both(float2 v, float2 &f, float2 &df) {
    const float2 one = pair_of(1.f), minus = pair_of(-1.f);
    if constexpr (ACT == DLC_ACTIVATION_RELU) {
        f = act_f2<ACT>(v);
        df = make_float2(v.x > 0.f ? 1.f : 0.f, v.y > 0.f ? 1.f : 0.f);
    } else if constexpr (ACT == DLC_ACTIVATION_SIGMOID) {
        f = logistic(v);
        df = mul2(f, fma2(f, minus, one));
    } else if constexpr (ACT == DLC_ACTIVATION_TANH) {
        f = act_f2<ACT>(v);
        df = fma2(mul2(f, minus), f, one);
    } else if constexpr (ACT == DLC_ACTIVATION_SILU) {  // p (1 + v (1 - p))
        const float2 p = logistic(v);
        f = mul2(v, p);
        df = mul2(p, fma2(v, fma2(p, minus, one), one));
    } else if constexpr (ACT == DLC_ACTIVATION_GELU) {  // v Phi(v); Phi(v) + v phi(v)
        const float2 e = gauss(v), p = gelu_phi(v, e);
        f = mul2(v, p);
        df = fma2(mul2(v, e), pair_of(0.39894228040143268f), p);
    } else {
        f = v;
        df = one;
    }
}

// Calls fn(std::integral_constant<int, ACT>) for a runtime activation.
template <typename Fn>
__device__ __forceinline__ void act_dispatch(int act, Fn fn) {
    switch (act) {
        case DLC_ACTIVATION_RELU: fn(std::integral_constant<int, DLC_ACTIVATION_RELU>{}); break;
        case DLC_ACTIVATION_SIGMOID: fn(std::integral_constant<int, DLC_ACTIVATION_SIGMOID>{}); break;
        case DLC_ACTIVATION_TANH: fn(std::integral_constant<int, DLC_ACTIVATION_TANH>{}); break;
        case DLC_ACTIVATION_SILU: fn(std::integral_constant<int, DLC_ACTIVATION_SILU>{}); break;
        case DLC_ACTIVATION_GELU: fn(std::integral_constant<int, DLC_ACTIVATION_GELU>{}); break;
        default: fn(std::integral_constant<int, DLC_ACTIVATION_IDENTITY>{}); break;
    }
}

}  // namespace dlc
