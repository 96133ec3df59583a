// quant_tokens.cuh -- activations to the operands of the 128-granular product:
// E4M3 codes with one fp32 scale for each 128 consecutive values of a token.
//
//   y = x[row]  or  silu(g) u,   s = max|y| / 448 (1 for an all-zero piece; with
//   FP8_QUANT_POW2 rounded up to a power of two),   q = E4M3(y / s)
//
// HBM-bound: 2 bytes read (gated: 4) and 1 written per value.  A warp takes 256
// columns of a row at a time, lane l the 16 bytes of columns 8l .. 8l+7, so the
// sixteen lanes of a half-warp hold one 128-value piece and its maximum takes
// four shuffles; U such units are loaded before the first is converted.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "quant_kernel.cuh"

namespace bsfp8 {

constexpr int QTOK_THREADS = 256;

struct QuantTokensArgs {
    const __nv_bfloat16 *x;   // rows of ldx values; gated: gate in [0, K), up in [K, 2K)
    const int32_t *rows;      // [M] source rows, or null
    uint8_t *q;               // [M, K]
    float *s;                 // [M, KB]
    int64_t ldx, x_rows, units;   // units: M * chunks
    int K, KB, chunks;        // chunks of 256 columns per row
};

// s rounded up to a power of two, at least 2^-126 (so that 1/s is exact).
__device__ __forceinline__ float pow2_up(float s) {
    return __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0x7F800000u);
}

// silu(gate) * up in fp32: the sigmoid from exp(-|gate|) <= 1, so that no
// exponential overflows and small results keep their relative precision.
__device__ __forceinline__ float silu_mul(float gate, float up) {
    const float e = expf(-fabsf(gate));
    const float r = __frcp_rn(1.0f + e);
    return gate * (gate >= 0.0f ? r : e * r) * up;
}

template <bool GATED, bool POW2, int U>
__global__ void __launch_bounds__(QTOK_THREADS) bsfp8_quantize_tokens(const QuantTokensArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (QTOK_THREADS / 32);
    const int64_t w0 = static_cast<int64_t>(blockIdx.x) * (QTOK_THREADS / 32) + (threadIdx.x >> 5);
    for (int64_t base = w0; base < a.units; base += warps * U) {
        uint4 v[U], up[GATED ? U : 1];
        int64_t row[U];
        int col[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t unit = base + u * warps;
            row[u] = unit / a.chunks;
            col[u] = static_cast<int>(unit - row[u] * a.chunks) * 256 + 8 * lane;
            in[u] = unit < a.units && col[u] < a.K;
            int64_t src = row[u];
            if (a.rows && in[u]) src = __ldg(a.rows + row[u]);
            const bool ok = in[u] && src >= 0 && src < a.x_rows;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            const __nv_bfloat16 *p = a.x + src * a.ldx + col[u];
            v[u] = ok ? __ldg(reinterpret_cast<const uint4 *>(p)) : zero;
            if constexpr (GATED) up[u] = ok ? __ldg(reinterpret_cast<const uint4 *>(p + a.K)) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            float y[8];
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[2 * j] = __uint_as_float(w[j] << 16);
                y[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
            if constexpr (GATED) {
                const uint32_t h[4] = {up[u].x, up[u].y, up[u].z, up[u].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[2 * j] = silu_mul(y[2 * j], __uint_as_float(h[j] << 16));
                    y[2 * j + 1] = silu_mul(y[2 * j + 1], __uint_as_float(h[j] & 0xFFFF0000u));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            if constexpr (GATED) {   // below the range of an exponential's fp32 precision: nothing
                if (!(amax >= 0x1p-100f)) amax = 0.0f;
                if (amax == 0.0f) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = 0.0f;
                }
            }
            float s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
            if constexpr (POW2) s = pow2_up(s);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(y[j], s);
            const uint2 codes = make_uint2(e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16,
                                           e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16);
            if (in[u]) {
                *reinterpret_cast<uint2 *>(a.q + row[u] * a.K + col[u]) = codes;
                if ((lane & 15) == 0) a.s[row[u] * a.KB + col[u] / 128] = s;
            }
        }
    }
}

}  // namespace bsfp8
