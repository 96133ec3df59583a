// epilogue.cuh -- bias, activation and residual applied to a product's fp32 sums before
// their one rounding to bf16:
//
//   C[m,n] = bf16( act(sum[m,n] + bias[n]) + R[m,n] )
//
// The activations are evaluated in fp32 on ex2.approx and rcp.approx (2 ulp each) and are
// off by less than 2^-14 relative wherever the result is a normal bf16 number, a thirtieth
// of the half step of the rounding that follows:
//   silu(y) = y s(y), gelu_tanh(y) = y s(2 sqrt(2/pi) (y + 0.044715 y^3)), s the logistic
//     function, from the exponential of the negative side only, so that nothing overflows and the
//     tail of negative y keeps its relative precision;
//   gelu(y) = y Phi(y), Phi the normal distribution's integral: Phi(-z) = 2^q(z) with q a
//     polynomial of degree 9, the minimax fit of log2 Phi(-z) on [0, 14.3] (beyond it Phi(-z)
//     is below the smallest fp32 number): in fp32 at most 4.2e-5 relative up to z = 6, 6.1e-5
//     (2^-14) up to z = 13.1, from where on the result is no normal bf16 number, and 8.7e-5
//     from there to 14.3; Phi(z) = 1 - Phi(-z).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace bsfp8 {

// FP8_ACT_* of bsfp8.h
enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

struct Epilogue {
    const void *bias;          // [N] fp32 or bf16, or null
    const __nv_bfloat16 *R;    // [M, N], or null; may be C
    int bias_bf16, act;
};

__device__ __forceinline__ float ex2(float x) {   // results below 2^-126 are 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {   // 1 <= x <= 2 here
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// y / (1 + 2^-2t), t = y (a + b y^2); silu: a = log2(e) / 2, b = 0; gelu_tanh: a = log2(e)
// sqrt(2/pi), b = 0.044715 a.  2^-2|t| is the square of n = 2^-|t|, so that the subnormal part of
// its range is there; y^2 is kept finite (b = 0 times infinity is NaN).  Each value has a reciprocal
// of its own: one for two of them, 1 / d0 = d1 / (d0 d1), takes a NaN and the last bits from one
// column to the next, and is no faster (4096^3 with bias, gelu_tanh and residual 86.6 us both ways).
// Written for scalar registers: packed pairs (f32x2) move the sums of the tile kernels' K loop
// about (19 % longer).
__device__ __forceinline__ float sigmoid_gate(float y, float a, float b) {
    const float t = y * fmaf(b, fminf(y * y, 1e30f), a), n = ex2(-fabsf(t));
    return y * ((t < 0.0f ? n * n : 1.0f) * rcp(fmaf(n, n, 1.0f)));
}

// The polynomial has 32 added, taken back after ex2, so that Phi may be a subnormal number; at
// z = 15 it is 0, however large y is.  On the positive side it is taken times z: 0 times +inf would
// be NaN (-inf gives that, as the formula does).
__device__ __forceinline__ float gelu(float y) {
    const float z = fminf(fabsf(y), 15.0f);
    float q = -0x1.98ee82p-30f;
    q = fmaf(q, z, 0x1.ee0552p-24f);
    q = fmaf(q, z, -0x1.052edcp-18f);
    q = fmaf(q, z, 0x1.3f86fcp-14f);
    q = fmaf(q, z, -0x1.f99df2p-11f);
    q = fmaf(q, z, 0x1.13c89ap-7f);
    q = fmaf(q, z, -0x1.b4e9e0p-5f);
    q = fmaf(q, z, -0x1.d69808p-2f);
    q = fmaf(q, z, -0x1.268e82p+0f);
    q = fmaf(q, z, 31.0f - 0x1.e6p-15f);
    const float tail = ex2(q) * 0x1p-32f;
    return y < 0.0f ? tail * y : fmaf(-tail, z, y);   // NaN stays NaN
}

// The activation of N values; one branch for all of them.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];   // NaN stays NaN
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gelu(v[i]);
    } else if (act != ACT_NONE) {
        const float a = act == ACT_SILU ? 0.5f * 1.44269504f : 0.5f * 2.30220819f;
        const float b = act == ACT_SILU ? 0.0f : 0.044715f * 0.5f * 2.30220819f;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = sigmoid_gate(v[i], a, b);
    }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// One value, of column n and place `at` in C (rows form).
__device__ __forceinline__ float finish(const Epilogue &e, float v, int n, int64_t at) {
    if (e.bias)
        v += e.bias_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(e.bias)[n])
                         : static_cast<const float *>(e.bias)[n];
    float one[1] = {v};
    activate(one, e.act);
    return e.R ? one[0] + __bfloat162float(e.R[at]) : one[0];
}

// Four values in a row: columns n .., a multiple of 4, of the row whose place in C is `at`.
__device__ __forceinline__ void finish4(const Epilogue &e, float (&v)[4], int n, int64_t at) {
    uint2 r = make_uint2(0u, 0u);
    if (e.R) r = *reinterpret_cast<const uint2 *>(e.R + at + n);
    if (e.bias) {
        if (e.bias_bf16) {
            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(e.bias) + n);
            v[0] += bf16_lo(w.x), v[1] += bf16_hi(w.x), v[2] += bf16_lo(w.y), v[3] += bf16_hi(w.y);
        } else {
            const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(e.bias) + n);
            v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
        }
    }
    activate(v, e.act);
    if (e.R) v[0] += bf16_lo(r.x), v[1] += bf16_hi(r.x), v[2] += bf16_lo(r.y), v[3] += bf16_hi(r.y);
}

}  // namespace bsfp8
