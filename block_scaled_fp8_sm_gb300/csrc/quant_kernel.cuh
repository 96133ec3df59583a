// quant_kernel.cuh -- block quantization of bf16 activations to the GEMM's
// operand format: E4M3 codes with one fp32 scale per 32x32 block, s = amax/448
// (1 for an all-zero block) and q = E4M3(x / s), nearest-even, saturating
// (FP8 GEMM library article, hncyxsy.com/news/241433, sections 2.1-2.2).
//
// HBM-bound: 2 bytes read and 1 byte written per element, plus 4 bytes per
// 1024 elements of scales.  One CTA of 256 threads covers a strip of 32 rows x
// 256 columns (eight blocks): warp w reads rows w, w+8, w+16 and w+24 of the
// strip, lane l the 16 bytes of columns 8l..8l+7, so every warp-row load is
// 512 contiguous bytes and every warp-row store 256.  Block b of the strip is
// held by lanes 4b..4b+3 of all eight warps: its maximum magnitude is taken on
// packed bf16 pairs, reduced over those four lanes with shuffles, then over the
// warps through shared memory.  Five CTAs stay resident per SM (48 registers).
//
// The arithmetic is quant_math.cuh's.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "quant_math.cuh"

namespace bsfp8 {

constexpr int QT_COLS = 256;
constexpr int QT_THREADS = 256;
constexpr int QT_MIN_CTAS = 5;   // resident CTAs per SM the register budget is set for

// Codes of the lane's four rows of the strip (the path is chosen once per strip).
template <bool RECIP>
__device__ __forceinline__ void store_codes(const uint32_t (&w)[4][4], float s, float nrc, uint8_t *q, int64_t r0,
                                            int64_t col, bool col_ok, int64_t M, int64_t K) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 8 * i;
        const uint2 out = codes8<RECIP>(w[i], s, nrc);
        if (col_ok && r < M) *reinterpret_cast<uint2 *>(q + r * K + col) = out;
    }
}

__global__ void __launch_bounds__(QT_THREADS, QT_MIN_CTAS) bsfp8_quantize_blocks(const __nv_bfloat16 *__restrict__ x,
                                                                                   uint8_t *__restrict__ q,
                                                                                   float *__restrict__ s, int64_t M,
                                                                                   int64_t K) {
    __shared__ float part[QT_THREADS / 32][QT_COLS / 32];   // [warp][block] maxima
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * QT_COLS + 8 * lane;
    const bool col_ok = col < K;   // K is a multiple of 32: 8-column groups are whole
    const int64_t MB = (M + 31) / 32, KB = K / 32;
    for (int64_t mb = blockIdx.y; mb < MB; mb += gridDim.y) {
        const int64_t r0 = mb * 32 + warp;
        uint32_t w[4][4];
        uint32_t am2 = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 8 * i;
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (col_ok && r < M) raw = *reinterpret_cast<const uint4 *>(x + r * K + col);
            w[i][0] = raw.x;
            w[i][1] = raw.y;
            w[i][2] = raw.z;
            w[i][3] = raw.w;
#pragma unroll
            for (int j = 0; j < 4; ++j) am2 = absmax_bf16x2(am2, w[i][j]);
        }
        float amax = fmaxf(__uint_as_float(am2 << 16), __uint_as_float(am2 & 0xFFFF0000u));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        if ((lane & 3) == 0) part[warp][lane >> 2] = amax;
        __syncthreads();
        float bmax = part[0][lane >> 2];
#pragma unroll
        for (int w8 = 1; w8 < QT_THREADS / 32; ++w8) bmax = fmaxf(bmax, part[w8][lane >> 2]);
        __syncthreads();   // part is rewritten by the next row block
        const float sc = block_scale(bmax);
        if (warp == 0 && (lane & 3) == 0 && col_ok) s[mb * KB + col / 32] = sc;
        if (sc >= 0x1p-100f && sc <= 3.40282347e38f)
            store_codes<true>(w, sc, -__frcp_rn(sc), q, r0, col, col_ok, M, K);
        else
            store_codes<false>(w, sc, 0.0f, q, r0, col, col_ok, M, K);
    }
}

}  // namespace bsfp8
