// block128_api.cu -- host side of the 128-granular entry points of
// include/bsfp8.h: argument checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "block128_rows.cuh"
#include "block128_native.cuh"
#include "block128_tile.cuh"
#include "bsfp8.h"
#include "host.h"
#include "quant_tokens.cuh"

namespace bsfp8 {

namespace {

template <int BN, bool SPLIT, bool FUSED>
int set_tile_attrs() {
    return cudaFuncSetAttribute(bsfp8_block128_tile<BN, SPLIT, FUSED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem128<BN, FUSED>()) == cudaSuccess
               ? FP8_OK
               : FP8_ERR_CUDA;
}

template <bool FUSED>
int set_attrs() {
    if (set_tile_attrs<256, false, FUSED>() != FP8_OK || set_tile_attrs<128, false, FUSED>() != FP8_OK ||
        set_tile_attrs<128, true, FUSED>() != FP8_OK)
        return FP8_ERR_CUDA;
    return cudaFuncSetAttribute(bsfp8_block128_native<FUSED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem_n128()) == cudaSuccess
               ? FP8_OK
               : FP8_ERR_CUDA;
}

}  // namespace

int block128_setup() {
    const int rc = set_attrs<false>();
    return rc != FP8_OK ? rc : set_attrs<true>();
}

namespace {

// Mode and sizes of both products.
int check_sizes(int64_t M, int64_t N, int64_t K, int mode) {
    if (mode != FP8_PATH_AUTO && mode != FP8_PATH_NATIVE && mode != FP8_PATH_PROMOTE) return FP8_ERR_MODE;
    if (M < 0 || N < 0 || K < 0 || M >= kLim || N >= kLim || K >= kLim) return FP8_ERR_SHAPE;
    return N % 8 != 0 || K % 16 != 0 ? FP8_ERR_SHAPE : FP8_OK;
}

// Their pointers, once there is something to compute.
int check_operands(const void *A, const float *sA, const void *B, const float *sB, const void *C, int64_t K) {
    if (!C) return FP8_ERR_NULL;
    if (!aligned(C, 16)) return FP8_ERR_ALIGN;
    if (K > 0) {
        if (!A || !B || !sA || !sB) return FP8_ERR_NULL;
        if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 4) || !aligned(sB, 4)) return FP8_ERR_ALIGN;
    }
    return FP8_OK;
}

// ONE_WAVE: the caller knows that all CTAs fit on the GPU at once.
template <int NT, int U, int WARPS, int CTAS, bool ONE_WAVE, bool FUSED>
int launch_rows(const RowsArgs &a, int64_t groups, DeviceState *d, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.N + ROWS_N - 1) / ROWS_N), static_cast<unsigned>(groups));
    if (ONE_WAVE || static_cast<int64_t>(grid.x) * groups <= static_cast<int64_t>(CTAS) * d->sm_count)
        return launch(bsfp8_block128_rows<NT, U, WARPS, CTAS, true, FUSED>, grid, WARPS * 32, 0, 1, a, stream);
    if constexpr (!ONE_WAVE)
        return launch(bsfp8_block128_rows<NT, U, WARPS, CTAS, false, FUSED>, grid, WARPS * 32, 0, 1, a, stream);
}

RowsArgs rows_args(const void *A, const float *sA, const void *B, const float *sB, void *C, int64_t M, int64_t N,
                   int64_t K) {
    RowsArgs a{};
    a.A = static_cast<const uint8_t *>(A);
    a.sA = sA;
    a.B = static_cast<const uint8_t *>(B);
    a.sB = sB;
    a.C = static_cast<__nv_bfloat16 *>(C);
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.KB = static_cast<int>((K + 127) / 128);
    return a;
}

int tile_args(Tile128Args &a, const RowsArgs &r, int BN, DeviceState *d) {
    const int64_t brows = static_cast<int64_t>(r.N) * (r.offsets ? r.E : 1);
    int rc = encode_kmajor(&a.tmA, r.A, r.M, r.K, T128_BM);
    if (rc != FP8_OK) return rc;
    rc = encode_kmajor(&a.tmA32, r.A, r.M, r.K, 32);
    if (rc != FP8_OK) return rc;
    rc = encode_kmajor(&a.tmB, r.B, brows, r.K, BN);
    if (rc != FP8_OK) return rc;
    a.sA = r.sA;
    a.sB = r.sB;
    a.C = r.C;
    a.offsets = r.offsets;
    a.status = d->status;
    a.wait_limit = wait_limit();
    a.withhold = withheld_stage();
    a.ep = r.ep;
    a.M = r.M;
    a.N = r.N;
    a.KB = r.KB;
    a.NB = (r.N + 127) / 128;
    a.E = r.E;
    a.mt = (r.M + T128_BM - 1) / T128_BM;
    a.nt = (r.N + BN - 1) / BN;
    // tile order: B passes once for each group of m-tiles, whose A is read from L2 then;
    // 32 MB is half of what one of the two L2 halves holds (8192 x 28672 x 8192, promotion /
    // native, runs of some ms: 32 MB 1406 / 1229 us, 16 MB 1396 / 1257, 64 MB 1496 / 1381)
    const int64_t fit = (int64_t(32) << 20) / (static_cast<int64_t>(T128_BM) * r.K);
    a.group = static_cast<int>(fit < 1 ? 1 : fit > a.mt ? a.mt : fit);
    return FP8_OK;
}

// `tiles`: how many there are, or, for experts, can be.
template <int BN, bool SPLIT, bool FUSED>
int launch_tile(const RowsArgs &r, int64_t tiles, int split, DeviceState *d, cudaStream_t stream) {
    Tile128Args a{};
    const int rc = tile_args(a, r, BN, d);
    if (rc != FP8_OK) return rc;
    // split: one tile per cluster; else persistent CTAs
    const int64_t ctas = SPLIT ? tiles * split : tiles < d->sm_count ? tiles : d->sm_count;
    return launch(bsfp8_block128_tile<BN, SPLIT, FUSED>, dim3(static_cast<unsigned>(ctas)), T128_THREADS,
                  smem128<BN, FUSED>(), split, a, stream);
}

template <bool FUSED>
int launch_native(const RowsArgs &r, int64_t tiles, DeviceState *d, cudaStream_t stream) {
    Tile128Args a{};
    const int rc = tile_args(a, r, N128_BN, d);
    if (rc != FP8_OK) return rc;
    const unsigned grid = static_cast<unsigned>(tiles < d->sm_count ? tiles : d->sm_count);
    return launch(bsfp8_block128_native<FUSED>, dim3(grid), T128_THREADS, smem_n128(), 1, a, stream);
}

// CTAs that share a tile's K: as many as the GPU still has room for, four K blocks
// each at least.
int split_of(int64_t tiles, int KB, int sms) {
    int split = 1;
    while (split < T128_MAX_SPLIT && tiles * split * 2 <= sms && KB >= split * 8) split *= 2;
    return split;
}

// The form of one product.
//
// Rows: up to 8 rows always (1 x 4096 x 7168 6.4 us against 9.2 by tiles, 1 x 28672 x 8192
// 37 against 47).  Up to 64 rows where B is small: the rows form costs about 2.3 us, and
// 0.24 us per MB of B for each group of 16 rows; tiles cost 5.6 us + 0.14 us per MB in all
// (16 x 4096 x 7168 9.3 / 9.2 us; 32 x 2048 x 4096 6.6 / 7.7; 64 x 1024 x 2048 4.3 / 7.0; 64
// x 8192 x 512 9.8 / 4.6).
//
// Tiles of 128 x 256 once they fill the SMs (4096^3 61 us; 72 with 128 columns), else of
// 128 x 128 with K split over clusters (37 x 4104 x 7184 10 us; 19 unsplit).
template <bool FUSED>
int launch_product(const RowsArgs &a, int mode, DeviceState *d, cudaStream_t stream) {
    const bool pinned = mode == FP8_PATH_PROMOTE;
    if (!pinned && a.M <= 8)
        return (a.N + ROWS_N - 1) / ROWS_N <= 2 * d->sm_count ? launch_rows<1, 4, 8, 2, true, FUSED>(a, 1, d, stream)
                                                              : launch_rows<1, 4, 4, 4, false, FUSED>(a, 1, d, stream);
    const int64_t groups = (a.M + 15) / 16;
    if (!pinned && groups <= 4 && static_cast<int64_t>(a.N) * a.K * (24 * groups - 14) <= 330000000ll)
        return (a.N + ROWS_N - 1) / ROWS_N * groups <= 2 * d->sm_count ? launch_rows<2, 1, 8, 2, true, FUSED>(a, groups, d, stream)
                                                                       : launch_rows<2, 2, 4, 4, false, FUSED>(a, groups, d, stream);
    const int64_t mt = (a.M + T128_BM - 1) / T128_BM;
    const int64_t wide = mt * ((a.N + 255) / 256), narrow = mt * ((a.N + 127) / 128);
    if (wide >= d->sm_count && mode == FP8_PATH_NATIVE) return launch_native<FUSED>(a, wide, d, stream);
    if (wide >= d->sm_count) return launch_tile<256, false, FUSED>(a, wide, 1, d, stream);
    const int split = pinned ? 1 : split_of(narrow, a.KB, d->sm_count);
    if (split > 1) return launch_tile<128, true, FUSED>(a, narrow, split, d, stream);
    return launch_tile<128, false, FUSED>(a, narrow, 1, d, stream);
}

// Experts: the row counts are on the device, so the rule goes by what is possible: at
// most min(E, T) + T / 128 row tiles.  Rows up to four on average (rows / tiles: 64 rows
// over 16 experts of 4096 x 7168 70 / 73 us, 96 rows 80 / 73; 32 over 8 of 1024 x 2048 4.9 /
// 7.5; 256 over 64 of 4096 x 2048 86 / 83, 384 97 / 84).  256-column tiles where they can
// fill the SMs (16 experts, 532 rows of 4096 x 7168: 77 us, 87 with 128 columns).
// Uneven routing costs the rows form more, as an expert's rows are taken eight at a time one
// after the other: all of them with one expert, against even, 195 / 264 us (256 rows over 64
// of 4096 x 7168), 164 / 93 (1024 over 256 of 1024 x 2048), 388 / 161 (4096 over 1024 of 512
// x 1024).  CTAs of their own for each 32 rows of an expert bring these to 113, 57 and 185,
// but cost even routing, whose grid then has rows for pieces that do not exist, up to 17 %
// (264, 96, 188).
int launch_experts(const RowsArgs &a, int mode, DeviceState *d, cudaStream_t stream) {
    const bool pinned = mode == FP8_PATH_PROMOTE;
    if (!pinned && a.M <= 4 * static_cast<int64_t>(a.E))
        return launch_rows<1, 2, 4, 6, false, false>(a, a.M < a.E ? a.M : a.E, d, stream);
    const int64_t most = (a.M < a.E ? a.M : a.E) + a.M / T128_BM;
    const int64_t wide = most * ((a.N + 255) / 256), narrow = most * ((a.N + 127) / 128);
    if (wide >= d->sm_count && mode == FP8_PATH_NATIVE) return launch_native<false>(a, wide, d, stream);
    if (wide >= d->sm_count) return launch_tile<256, false, false>(a, wide, 1, d, stream);
    const int split = pinned ? 1 : split_of(narrow, a.KB, d->sm_count);
    if (split > 1) return launch_tile<128, true, false>(a, narrow, split, d, stream);
    return launch_tile<128, false, false>(a, narrow, 1, d, stream);
}

template <bool GATED>
int quantize(const void *x, int64_t ldx, int64_t x_rows, const int32_t *rows, void *q, float *s, int64_t M,
             int64_t K, int flags, cudaStream_t stream) {
    const int64_t width = GATED ? 2 * K : K;
    if (M < 0 || K < 0 || x_rows < 0 || M >= kLim || width >= kLim || x_rows >= kLim || ldx >= 2 * kLim) return FP8_ERR_SHAPE;
    if (K % 16 != 0 || ldx < width || ldx % 8 != 0) return FP8_ERR_SHAPE;
    if (flags & ~FP8_QUANT_POW2) return FP8_ERR_MODE;
    if (M == 0 || K == 0) return FP8_OK;
    if (!q || !s || (!x && x_rows > 0)) return FP8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4) || !aligned(rows, 4)) return FP8_ERR_ALIGN;
    if (!rows && x_rows < M) return FP8_ERR_SHAPE;
    DeviceState *d = nullptr;
    const int rc = device_setup(&d);
    if (rc != FP8_OK) return rc;
    QuantTokensArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.rows = rows;
    a.q = static_cast<uint8_t *>(q);
    a.s = s;
    a.ldx = static_cast<uint32_t>(ldx);
    a.x_rows = static_cast<uint32_t>(x_rows);
    a.K = static_cast<uint32_t>(K);
    a.KB = static_cast<uint32_t>((K + 127) / 128);
    // p / KB for p < 2^31: multiplier ceil(2^(31 + l) / KB) with l = ceil(log2 KB)
    // (Granlund and Montgomery, PLDI 1994), below 2^32
    int l = 0;
    while ((int64_t(1) << l) < a.KB) ++l;
    a.shift = static_cast<uint32_t>(31 + l);
    a.mul = static_cast<uint32_t>(((uint64_t(1) << a.shift) + a.KB - 1) / a.KB);
    const int64_t step = (kLim * 2 - 1) / a.KB;   // rows per launch: fewer than 2^31 pieces
    for (int64_t m = 0; m < M; m += step) {
        const int64_t n = M - m < step ? M - m : step;
        a.pieces = static_cast<uint32_t>(n * a.KB);
        const int64_t ctas = (n * a.KB + QTOK_GROUPS - 1) / QTOK_GROUPS;
        const int64_t most = static_cast<int64_t>(d->sm_count) * 64;
        const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
        const int rc = launch(flags & FP8_QUANT_POW2 ? bsfp8_quantize_tokens<GATED, true>
                                                     : bsfp8_quantize_tokens<GATED, false>,
                              dim3(grid), QTOK_THREADS, 0, 1, a, stream);
        if (rc != FP8_OK) return rc;
        if (rows) {
            a.rows += n;
        } else {
            a.x += n * ldx;
            a.x_rows -= static_cast<uint32_t>(n);
        }
        a.q += n * K;
        a.s += n * a.KB;
    }
    return FP8_OK;
}

}  // namespace
}  // namespace bsfp8

using namespace bsfp8;

extern "C" {

int fp8_gemm_block128_ex(const void *A, const float *sA, const void *B, const float *sB, void *C, int64_t M,
                         int64_t N, int64_t K, int mode, cudaStream_t stream) {
    int rc = check_sizes(M, N, K, mode);
    if (rc != FP8_OK || M == 0 || N == 0) return rc;
    rc = check_operands(A, sA, B, sB, C, K);
    if (rc != FP8_OK) return rc;
    DeviceState *d = nullptr;
    rc = device_setup(&d);
    if (rc != FP8_OK) return rc;
    if (K == 0) return zero_fill(C, M * N, stream);
    RowsArgs a = rows_args(A, sA, B, sB, C, M, N, K);
    a.status = d->status;
    return guarded([&] { return launch_product<false>(a, mode, d, stream); });
}

int fp8_gemm_block128(const void *A, const float *sA, const void *B, const float *sB, void *C, int64_t M, int64_t N,
                      int64_t K, cudaStream_t stream) {
    return fp8_gemm_block128_ex(A, sA, B, sB, C, M, N, K, FP8_PATH_AUTO, stream);
}

int fp8_gemm_block128_fused(const void *A, const float *sA, const void *B, const float *sB, const void *bias,
                            int bias_type, int act, const void *R, void *C, int64_t M, int64_t N, int64_t K, int mode,
                            cudaStream_t stream) {
    int rc = check_sizes(M, N, K, mode);
    if (rc != FP8_OK) return rc;
    if ((bias_type != FP8_TYPE_F32 && bias_type != FP8_TYPE_BF16) || act < FP8_ACT_NONE || act > FP8_ACT_SILU)
        return FP8_ERR_MODE;
    if (M == 0 || N == 0) return FP8_OK;
    rc = check_operands(A, sA, B, sB, C, K);
    if (rc != FP8_OK) return rc;
    if (!aligned(bias, 16) || !aligned(R, 16)) return FP8_ERR_ALIGN;
    DeviceState *d = nullptr;
    rc = device_setup(&d);
    if (rc != FP8_OK) return rc;
    RowsArgs a = rows_args(A, sA, B, sB, C, M, N, K);
    a.status = d->status;
    a.ep = Epilogue{bias, static_cast<const __nv_bfloat16 *>(R), bias_type == FP8_TYPE_BF16, act};
    if (K > 0) return guarded([&] { return launch_product<true>(a, mode, d, stream); });
    // no K: act(bias) + R by the rows form, whose loops over K are then empty; up to 65535 groups a launch
    for (int64_t m = 0; m < M && rc == FP8_OK; m += 8 * 65535) {
        a.M = static_cast<int>(M - m < 8 * 65535 ? M - m : 8 * 65535);
        rc = launch_rows<1, 4, 4, 4, false, true>(a, (a.M + 7) / 8, d, stream);
        a.C += static_cast<int64_t>(a.M) * N;
        if (R) a.ep.R += static_cast<int64_t>(a.M) * N;
    }
    return rc;
}

int fp8_gemm_experts_ex(const void *A, const float *sA, const void *B, const float *sB, void *C,
                        const int32_t *offsets, int64_t T, int64_t N, int64_t K, int32_t E, int mode,
                        cudaStream_t stream) {
    if (E < 0 || E > FP8_MAX_EXPERTS || (N > 0 && N < kLim && E * N >= 2 * kLim)) return FP8_ERR_SHAPE;
    int rc = check_sizes(T, N, K, mode);
    if (rc != FP8_OK || T == 0 || N == 0 || E == 0) return rc;   // without experts the weights are no memory at all
    rc = check_operands(A, sA, B, sB, C, K);
    if (rc != FP8_OK) return rc;
    if (!offsets) return FP8_ERR_NULL;
    if (!aligned(offsets, 4)) return FP8_ERR_ALIGN;
    if (K == 0) return FP8_ERR_SHAPE;   // which rows belong to an expert is known on the device only
    DeviceState *d = nullptr;
    rc = device_setup(&d);
    if (rc != FP8_OK) return rc;
    RowsArgs a = rows_args(A, sA, B, sB, C, T, N, K);
    a.offsets = offsets;
    a.E = E;
    a.status = d->status;
    return guarded([&] { return launch_experts(a, mode, d, stream); });
}

int fp8_gemm_experts(const void *A, const float *sA, const void *B, const float *sB, void *C, const int32_t *offsets,
                     int64_t T, int64_t N, int64_t K, int32_t E, cudaStream_t stream) {
    return fp8_gemm_experts_ex(A, sA, B, sB, C, offsets, T, N, K, E, FP8_PATH_AUTO, stream);
}

int fp8_quantize_tokens(const void *x, int64_t ldx, int64_t x_rows, const int32_t *rows, void *q, float *s,
                        int64_t M, int64_t K, int flags, cudaStream_t stream) {
    return quantize<false>(x, ldx, x_rows, rows, q, s, M, K, flags, stream);
}

int fp8_swiglu_quantize_tokens(const void *x, int64_t ldx, void *q, float *s, int64_t M, int64_t K, int flags,
                               cudaStream_t stream) {
    return quantize<true>(x, ldx, M, nullptr, q, s, M, K, flags, stream);
}

}  // extern "C"
