// epilogue.cuh -- bias, activation and residual applied to a product's fp32 sums before
// their one rounding to bf16:
//
//   C[m,n] = bf16( act(sum[m,n] + bias[n]) + R[m,n] )
//
// The activations are evaluated in fp32 on ex2.approx and rcp.approx (2 ulp each) and are
// off by less than 2^-14 relative wherever the result is a normal bf16 number, a thirtieth
// of the half step of the rounding that follows:
//   silu(y)      = y s(y log2(e)), gelu_tanh(y) = y s(2 log2(e) sqrt(2/pi) (y + 0.044715 y^3)),
//     s(t) = 1 / (1 + 2^-t), from 2^-|t| only, so that nothing overflows and the tail of
//     negative y keeps its relative precision;
//   gelu(y)      = y Phi(y), Phi the normal distribution's integral: Phi(-z) = 2^q(z) with
//     q a polynomial of degree 9, the minimax fit of log2 Phi(-z) on [0, 14.3] (beyond it
//     Phi(-z) is below the smallest fp32 number): at most 4.2e-5 relative up to z = 6 and
//     8.8e-5 after; Phi(z) = 1 - Phi(-z).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace bsfp8 {

// FP8_ACT_* of bsfp8.h
enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

struct Epilogue {
    const void *bias;          // [N] fp32 or bf16, or null
    const __nv_bfloat16 *R;    // [M, N], or null; may be C
    int bias_bf16, act;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// y / (1 + 2^-t)
__device__ __forceinline__ float times_sigmoid2(float y, float t) {
    const float e = ex2(-fabsf(t)), r = rcp(1.0f + e);
    return y * (t < 0.0f ? e * r : r);
}

__device__ __forceinline__ float silu(float y) { return times_sigmoid2(y, y * 1.44269504f); }

__device__ __forceinline__ float gelu_tanh(float y) {
    constexpr float k = 2.30220819f;   // 2 log2(e) sqrt(2/pi)
    return times_sigmoid2(y, y * fmaf(k * 0.044715f, y * y, k));
}

__device__ __forceinline__ float gelu(float y) {
    const float z = fminf(fabsf(y), 14.3f);
    float q = -0x1.98ee82p-30f;
    q = fmaf(q, z, 0x1.ee0552p-24f);
    q = fmaf(q, z, -0x1.052edcp-18f);
    q = fmaf(q, z, 0x1.3f86fcp-14f);
    q = fmaf(q, z, -0x1.f99df2p-11f);
    q = fmaf(q, z, 0x1.13c89ap-7f);
    q = fmaf(q, z, -0x1.b4e9e0p-5f);
    q = fmaf(q, z, -0x1.d69808p-2f);
    q = fmaf(q, z, -0x1.268e82p+0f);
    q = fmaf(q, z, -0x1.0003ccp+0f);
    const float p = ex2(q) * y;        // NaN stays NaN by y
    return y < 0.0f ? p : y - p;
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
    } else if (act == ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gelu_tanh(v[i]);
    } else if (act == ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = silu(v[i]);
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
    if (e.R) one[0] += __bfloat162float(e.R[at]);
    return one[0];
}

// N (4 or 8) values in a row: columns n .., a multiple of N, with the residual's words r.
template <int N>
__device__ __forceinline__ void finish(const Epilogue &e, float (&v)[N], int n, const uint32_t (&r)[N / 2]) {
    if (e.bias) {
        if (e.bias_bf16) {
            const uint32_t *b = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(e.bias) + n);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const uint32_t w = b[i];
                v[2 * i] += bf16_lo(w);
                v[2 * i + 1] += bf16_hi(w);
            }
        } else {
            const float4 *b = reinterpret_cast<const float4 *>(static_cast<const float *>(e.bias) + n);
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 w = b[i];
                v[4 * i] += w.x;
                v[4 * i + 1] += w.y;
                v[4 * i + 2] += w.z;
                v[4 * i + 3] += w.w;
            }
        }
    }
    activate(v, e.act);
    if (e.R) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            v[2 * i] += bf16_lo(r[i]);
            v[2 * i + 1] += bf16_hi(r[i]);
        }
    }
}

}  // namespace bsfp8
