// quant_tokens.cuh -- activations to the operands of the 128-granular product:
// E4M3 codes with one fp32 scale for each 128 consecutive values of a token.
//
//   y = x[row]  or  silu(g) u,   s = max|y| / 448 (1 for an all-zero piece; with
//   FP8_QUANT_POW2 rounded up to a power of two),   q = E4M3(y / s)
//
// 2 bytes read (gated: 4) and 1 written per value: HBM sets the floor, and a value
// may cost few instructions before the integer and conversion pipes set the time.
// So eight lanes share a piece, sixteen values each (columns 8l .. 8l+7 and 64 + 8l ..
// of the piece: every load of a warp is four runs of 128 bytes): the maximum takes
// three shuffles for sixteen values.  The row of a piece comes from a multiplication
// by the reciprocal of the pieces per row.  Loads in flight come from resident warps (64
// of them an SM, 48 where the arithmetic needs 40 registers), not from pieces loaded ahead:
// 16384 x 7168 gathered from 4096 tokens 36.6 us alone, 39 in a loop over other inputs (180
// MB at the copy bandwidth 27; L2 serves the repeated tokens), all distinct 52 us (53),
// gated 16001 x 4096 58.0 us in such a loop (49: integer and conversion work); two pieces
// ahead with half the warps 41 / 57 / 65.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "block128_rows.cuh"
#include "quant_math.cuh"

namespace bsfp8 {

constexpr int QTOK_THREADS = 256;
constexpr int QTOK_GROUPS = QTOK_THREADS / 8;   // pieces a CTA converts at a time

struct QuantTokensArgs {
    const __nv_bfloat16 *x;   // rows of ldx values; gated: gate in [0, K), up in [K, 2K)
    const int32_t *rows;      // [M] source rows, or null
    uint8_t *q;               // [M, K]
    float *s;                 // [M, KB]
    uint32_t ldx, x_rows;     // (32-bit factors: one wide multiplication per address)
    uint32_t pieces;          // M * KB < 2^31
    uint32_t mul, shift;      // piece / KB = piece * mul >> shift, exact for pieces < 2^31
    uint32_t K, KB;
};

// s rounded up to a power of two, at least 2^-126 (so that 1/s is exact).
__device__ __forceinline__ float pow2_up(float s) {
    return __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0x7F800000u);
}

// silu(g) u on two values.  exp(-|g|) = 2^t, t = -|g| log2(e): the product's rounding
// error comes from an fma (Dekker's error-free product) and enters as 2^t (1 + t_lo ln 2);
// the sigmoid is r = 1 / (1 + e), or e r for negative g, so no exponential overflows.
// |g| counts as at most 256, whose exponential is zero, so that the product stays finite.
// Gates of kDeep and below are silu_mul2_deep's.
__device__ __forceinline__ uint64_t silu_mul2(uint64_t g, uint64_t u) {
    constexpr float kL = 0x1.715476p+0f, kLlo = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;   // log2(e) = kL + kLlo
    uint32_t g0, g1;
    f32x2_unpack(g, g0, g1);
    const uint64_t a = f32x2_of(fminf(fabsf(__uint_as_float(g0)), 256.0f), fminf(fabsf(__uint_as_float(g1)), 256.0f));
    const uint64_t t = mul_f32x2_rn(a, f32x2_of(-kL, -kL));
    uint64_t lo = fma_f32x2_rn(a, f32x2_of(kL, kL), t);   // |g| log2(e) + t = -t_lo
    lo = fma_f32x2_rn(a, f32x2_of(kLlo, kLlo), lo);
    uint32_t t0, t1;
    f32x2_unpack(t, t0, t1);
    float e0, e1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(__uint_as_float(t0)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(__uint_as_float(t1)));
    uint64_t e = f32x2_of(e0, e1);
    e = fma_f32x2_rn(mul_f32x2_rn(lo, f32x2_of(-kLn2, -kLn2)), e, e);
    uint32_t b0, b1;
    f32x2_unpack(e, b0, b1);
    float r0, r1;
    const float d0 = 1.0f + __uint_as_float(b0), d1 = 1.0f + __uint_as_float(b1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
    uint64_t r = f32x2_of(r0, r1);
    const uint32_t n0 = static_cast<int32_t>(g0) < 0 ? b0 : 0x3F800000u;   // e for negative g, else 1
    const uint32_t n1 = static_cast<int32_t>(g1) < 0 ? b1 : 0x3F800000u;
    const uint64_t sig = mul_f32x2_rn(f32x2_pack(n0, n1), r);
    return mul_f32x2_rn(mul_f32x2_rn(g, sig), u);
}

constexpr float kDeep = -64.0f;

// The same for g <= kDeep: y of the values above it stays.  exp(g) gets subnormal from -87
// on, and u may bring the result back into range, so each factor takes one half of the
// exponent: with n = 2^(t / 2), y = (g n) (u n) (the sigmoid is n^2: 1 + n^2 rounds to 1).
// |g n| < 1, so u n is larger than the result and has its bits as long as that is normal.
__device__ __forceinline__ uint64_t silu_mul2_deep(uint64_t y, uint64_t g, uint64_t u) {
    constexpr float kH = 0x1.715476p-1f, kHlo = 0x1.4ae0cp-27f, kLn2 = 0x1.62e43p-1f;   // log2(e) / 2 = kH + kHlo
    uint32_t gw[2], uw[2], yw[2];
    f32x2_unpack(g, gw[0], gw[1]);
    f32x2_unpack(u, uw[0], uw[1]);
    f32x2_unpack(y, yw[0], yw[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float gk = __uint_as_float(gw[k]), a = fminf(fabsf(gk), 256.0f);
        const float t = a * -kH, lo = fmaf(a, kHlo, fmaf(a, kH, t));
        float n;
        asm("ex2.approx.f32 %0, %1;" : "=f"(n) : "f"(t));
        n = fmaf(lo * -kLn2, n, n);
        if (gk <= kDeep) yw[k] = __float_as_uint((gk * n) * (__uint_as_float(uw[k]) * n));
    }
    return f32x2_pack(yw[0], yw[1]);
}

// The lesser value of each half.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The E4M3 codes of eight values, in order.
__device__ __forceinline__ uint2 pack_codes(const float (&v)[8]) {
    return make_uint2(__byte_perm(e4m3x2(v[0], v[1]), e4m3x2(v[2], v[3]), 0x5410),
                      __byte_perm(e4m3x2(v[4], v[5]), e4m3x2(v[6], v[7]), 0x5410));
}

// Codes of y / s for eight fp32 values (packed pairs): the quotient by the
// correctly rounded reciprocal and its remainder, negated as in codes8.
__device__ __forceinline__ uint2 codes8_f32(const uint64_t (&y)[4], float s, float nrc) {
    const uint64_t n2 = f32x2_of(nrc, nrc), s2 = f32x2_of(s, s);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t q = mul_f32x2_rn(y[j], n2);
        uint32_t lo, hi;
        f32x2_unpack(fma_f32x2_rn(fma_f32x2_rn(q, s2, y[j]), n2, q), lo, hi);
        v[2 * j] = __uint_as_float(lo);
        v[2 * j + 1] = __uint_as_float(hi);
    }
    const uint2 c = pack_codes(v);
    return make_uint2(c.x ^ 0x80808080u, c.y ^ 0x80808080u);
}

// Codes of y * inv, inv an exact power of two.
__device__ __forceinline__ uint2 codes8_pow2(const uint64_t (&y)[4], float inv) {
    const uint64_t i2 = f32x2_of(inv, inv);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        f32x2_unpack(mul_f32x2_rn(y[j], i2), lo, hi);
        v[2 * j] = __uint_as_float(lo);
        v[2 * j + 1] = __uint_as_float(hi);
    }
    return pack_codes(v);
}

template <bool GATED, bool POW2>
__global__ void __launch_bounds__(QTOK_THREADS, GATED || !POW2 ? 6 : 8) bsfp8_quantize_tokens(const QuantTokensArgs a) {
    launch_dependents();
    wait_for_previous();
    const uint32_t l = threadIdx.x & 7u;
    const uint32_t stride = gridDim.x * QTOK_GROUPS;
    // the whole warp stays in the loop together (shuffles): the bound is the warp's
    const uint32_t first = blockIdx.x * QTOK_GROUPS + (threadIdx.x >> 5) * 4, mine = (threadIdx.x >> 3) & 3;
    for (uint32_t base = first; base < a.pieces; base += stride) {
        uint4 v[2], up[2];
        const uint32_t p = base + mine;
        const bool in = p < a.pieces;
        const uint32_t row = static_cast<uint32_t>(static_cast<uint64_t>(p) * a.mul >> a.shift);
        const uint32_t kb = p - row * a.KB;
        const uint32_t col = kb * 128u + 8u * l;   // and col + 64
        uint32_t src = row;
        if (a.rows && in) src = static_cast<uint32_t>(a.rows[row]);   // a negative index is a large one
        const bool ok = in && src < a.x_rows;
        const __nv_bfloat16 *px = a.x + (static_cast<uint64_t>(src) * a.ldx + col);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool there = ok && col + 64u * j < a.K;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            v[j] = there ? *reinterpret_cast<const uint4 *>(px + 64 * j) : zero;
            if constexpr (GATED) up[j] = there ? *reinterpret_cast<const uint4 *>(px + a.K + 64 * j) : zero;
        }
        uint32_t w[2][4];
        uint64_t y[2][4];
        float amax;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            w[j][0] = v[j].x;
            w[j][1] = v[j].y;
            w[j][2] = v[j].z;
            w[j][3] = v[j].w;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[j][i] = f32x2_pack(w[j][i] << 16, w[j][i] & 0xFFFF0000u);
        }
        if constexpr (GATED) {
            amax = 0.0f;
            // the warp's least gate decides whether deep values are looked for (a value's bits do
            // not depend on it; doing without a branch, both factors with half of the exponent
            // everywhere, took 60.6 us and doubled the exponential's error)
            uint32_t least = min_bf16x2(w[0][0], w[1][0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) least = min_bf16x2(least, min_bf16x2(w[0][i], w[1][i]));
            const float lowest = fminf(__uint_as_float(least << 16), __uint_as_float(least & 0xFFFF0000u));
            const bool deep = __any_sync(0xFFFFFFFFu, lowest <= kDeep);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t h[4] = {up[j].x, up[j].y, up[j].z, up[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t g = y[j][i], u = f32x2_pack(h[i] << 16, h[i] & 0xFFFF0000u);
                    y[j][i] = silu_mul2(g, u);
                    if (deep) y[j][i] = silu_mul2_deep(y[j][i], g, u);
                    uint32_t lo, hi;
                    f32x2_unpack(y[j][i], lo, hi);
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(lo)), fabsf(__uint_as_float(hi))));
                }
            }
        } else {
            uint32_t am2 = 0u;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) am2 = absmax_bf16x2(am2, w[j][i]);
            amax = fmaxf(__uint_as_float(am2 << 16), __uint_as_float(am2 & 0xFFFF0000u));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        float s, f;
        uint2 codes[2];
        if constexpr (GATED) {
            const bool none = !(amax >= 0x1p-100f);   // below: the piece counts as all zero
            s = block_scale(none ? 0.0f : amax);
            if constexpr (POW2) s = pow2_up(s);
            f = none ? 0.0f : POW2 ? __frcp_rn(s) : -__frcp_rn(s);
            if (none) {
                codes[0] = codes[1] = make_uint2(0u, 0u);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    // an infinite scale (y past the largest fp32 number): f is zero, and a finite factor
                    // in the remainder leaves 0 for finite y and NaN for infinite ones
                    codes[j] = POW2 ? codes8_pow2(y[j], f) : codes8_f32(y[j], fminf(s, 3.40282347e38f), f);
            }
        } else if constexpr (POW2) {
            s = pow2_up(block_scale(amax));
            f = __uint_as_float(0x7F000000u - __float_as_uint(s));   // 1 / s
#pragma unroll
            for (int j = 0; j < 2; ++j) codes[j] = codes8_pow2(y[j], f);
        } else {
            s = block_scale(amax);
            const bool recip = s >= 0x1p-100f && s <= 3.40282347e38f;
            if (recip) {
                f = -__frcp_rn(s);
#pragma unroll
                for (int j = 0; j < 2; ++j) codes[j] = codes8<true>(w[j], s, f);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) codes[j] = codes8<false>(w[j], s, 0.0f);
            }
        }
        if (in) {
            uint8_t *pq = a.q + (static_cast<uint64_t>(row) * a.K + col);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (col + 64u * j < a.K) *reinterpret_cast<uint2 *>(pq + 64 * j) = codes[j];
            if (l == 0) a.s[p] = s;
        }
    }
}

}  // namespace bsfp8
