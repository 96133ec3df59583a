// quant_math.cuh -- the quantizers' arithmetic: scales s = amax/448 (1 for an all-zero
// group) and codes q = E4M3(x / s), nearest-even, saturating.
//
// A quantizer is bound by its integer/logic pipe rather than by HBM once the
// per-element work is a division, so the arithmetic is kept to a few packed
// instructions per element pair:
//   * s = RN(amax/448) as RN(y + RN(amax - 448 y) / 448) with y = RN(amax r),
//     r = RN(1/448) -- Markstein's correction (P. Markstein, IBM J. Res.
//     Develop. 34(1), 1990) -- equal to the correctly rounded division for
//     every positive finite bf16 amax (checked by enumeration);
//   * x/s from one reciprocal rc = RN(1/s) per block with the same correction,
//     evaluated on -x/s so that no operand needs negating in the packed f32x2
//     form: y' = RN(x (-rc)), e = RN(x + y' s), n = RN(y' + e (-rc)) = -RN(x/s)
//     wherever the residual e is exact; the E4M3 code of -v is the code of v
//     with bit 7 flipped, so the codes are XORed with 0x80.  Enumerating every
//     positive bf16 amax and every bf16 x with |x| <= amax shows that for
//     scales s >= 2^-100 the result equals RN(x/s) wherever |x/s| >= 2^-10 and
//     every code equals that of the correctly rounded division (below 2^-10
//     both codes are +-0).  Smaller or non-finite scales divide (x by -s).
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace bsfp8 {

// Two fp32 values -> two E4M3 codes (nearest-even, saturating), lo in byte 0.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Running maximum of |x| over packed bf16 pairs (maxNum: a NaN operand is
// ignored, as the oracle's comparison ignores it).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t acc, uint32_t w) {
    uint32_t a, d;
    asm("abs.bf16x2 %0, %1;" : "=r"(a) : "r"(w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(acc), "r"(a));
    return d;
}

// s = amax / 448 correctly rounded (1 for an all-zero block; an infinite
// maximum keeps s = inf, as the division gives).
__device__ __forceinline__ float block_scale(float amax) {
    constexpr float kR448 = 0x1.24924ap-9f;   // RN(1/448)
    const float y = __fmul_rn(amax, kR448);
    const float s = __fmaf_rn(__fmaf_rn(-y, 448.0f, amax), kR448, y);
    return amax > 0.0f ? (amax <= 3.40282347e38f ? s : amax) : 1.0f;
}

// The 8 codes of one lane's row segment: word j holds columns 2j (low half)
// and 2j+1 (high half).  RECIP: finite s >= 2^-100 with nrc = -RN(1/s).
template <bool RECIP>
__device__ __forceinline__ uint2 codes8(const uint32_t (&w)[4], float s, float nrc) {
    float v[8];
    if constexpr (RECIP) {
        const uint64_t nr2 = f32x2_pack(__float_as_uint(nrc), __float_as_uint(nrc));
        const uint64_t s2 = f32x2_pack(__float_as_uint(s), __float_as_uint(s));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t x2 = f32x2_pack(w[j] << 16, w[j] & 0xFFFF0000u);
            const uint64_t y2 = mul_f32x2_rn(x2, nr2);    // -y
            const uint64_t e2 = fma_f32x2_rn(y2, s2, x2);  // x - y s
            uint32_t lo, hi;
            f32x2_unpack(fma_f32x2_rn(e2, nr2, y2), lo, hi);   // -(y + e r)
            v[2 * j] = __uint_as_float(lo);
            v[2 * j + 1] = __uint_as_float(hi);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __fdiv_rn(__uint_as_float(w[j] << 16), -s);
            v[2 * j + 1] = __fdiv_rn(__uint_as_float(w[j] & 0xFFFF0000u), -s);
        }
    }
    return make_uint2(__byte_perm(e4m3x2(v[0], v[1]), e4m3x2(v[2], v[3]), 0x5410) ^ 0x80808080u,
                      __byte_perm(e4m3x2(v[4], v[5]), e4m3x2(v[6], v[7]), 0x5410) ^ 0x80808080u);
}

// One 32 x 32 block held by a warp, one row per lane: the lane's 32 bf16 values
// in bf[16] (columns 2j and 2j+1 in word j).  Returns the block's scale (its
// maximum over all 32 lanes) and leaves the lane's 32 codes in codes[8] (byte b
// of word w: column 4w + b) -- the quantizer's arithmetic above, so the codes
// and scale equal those of fp8_quantize_blocks on the same bf16 values.  Every
// lane of the warp must call it (shuffles); rows that do not exist pass zeros.
__device__ __forceinline__ float quantize_rows32(const uint32_t (&bf)[16], uint32_t (&codes)[8]) {
    uint32_t am2 = 0u;
#pragma unroll
    for (int j = 0; j < 16; ++j) am2 = absmax_bf16x2(am2, bf[j]);
    float amax = fmaxf(__uint_as_float(am2 << 16), __uint_as_float(am2 & 0xFFFF0000u));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    const float sc = block_scale(amax);
    const bool recip = sc >= 0x1p-100f && sc <= 3.40282347e38f;   // the same for the whole warp
    const float nrc = recip ? -__frcp_rn(sc) : 0.0f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint32_t w[4] = {bf[4 * g], bf[4 * g + 1], bf[4 * g + 2], bf[4 * g + 3]};
        const uint2 cc = recip ? codes8<true>(w, sc, nrc) : codes8<false>(w, sc, 0.0f);
        codes[2 * g] = cc.x;
        codes[2 * g + 1] = cc.y;
    }
    return sc;
}

}  // namespace bsfp8
