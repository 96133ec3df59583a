// block128_rows.cuh -- the 128-granular product for few rows of A.
//
//   C[m,n] = bf16( sum_kb sA[m][kb] sB[n/128][kb] sum_{k in kb} A[m,k] B[n,k] )
//
// With few rows the call is bound by reading B once (N K bytes) and by latency,
// not by the tensor cores, so there is no staging: a CTA of WARPS (four or eight)
// warps owns 16 rows of B and all of K, warp w taking the K blocks w, w + WARPS, ...
// and loading U of them ahead; each lane loads 16-byte pieces of B (and of the tokens) straight into registers, which
// are the operands of mma.m16n8k32 (B's 16 rows as its M side, 8 tokens as its
// N side).  The products of a 128-K block are summed by four MMAs from zero in
// fp32, then acc += (sA sB) * sum in fp32; the warps' sums are added in
// warp order.  A row's bits do not depend on the other rows.
//
// What bounds a launch is how many bytes of B are on their way.  Up to two CTAs for each
// SM (4096 columns: 256): eight warps, U = 4 blocks loaded ahead, two CTAs on an SM (1 x
// 4096 x 7168, weights not in L2: 8.3 us; U = 2 and three CTAs 9.2, four warps 9.4; in L2
// 6.4).  More CTAs: four warps, U = 4, four CTAs on an SM (8 x 16384 x 8192 25.0 us, 5.4
// TB/s; the former 28.5, U = 2 and eight warps 26.8).  Experts, where each CTA first finds
// its expert: four warps, U = 2, six CTAs, whose loads cover one another's starts (24 rows
// over 64 experts of 4096 x 7168: 85.7 us, 6.5 TB/s; U = 4 and four CTAs 90; eight CTAs of
// 64 registers 89).  Two groups of tokens (NT = 2) take twice the registers for them: eight
// warps, U = 1 and two CTAs on an SM (16 x 4096 x 7168, cold, 10.3 us; three CTAs 14.6), or
// four warps, U = 2 and four CTAs (16 x 16384 x 1024 6.4 us; the former 7.4).
//
// Every launch may be set up while the previous kernel ends (programmatic dependent
// launch); NEXT, a launch whose CTAs all fit on the GPU at once (one token: 256), also lets
// the next one in after its K loop: 1 x 4096 x 7168 in a stream of calls 8.2 -> 6.4 us.  At
// its start the next launch's CTAs would take its places on the SMs (7.6 us), and launches
// of several waves lose by it (24 rows over 64 experts 89 -> 115 us).
//
// The K order inside a block is permuted alike on both sides: lane t of a
// quad holds bytes 64 j + 16 t .. + 15 (j = 0, 1), so a load of a warp covers 64
// contiguous bytes of each of 8 rows.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"
#include "status.h"

namespace bsfp8 {

struct RowsArgs {
    const uint8_t *A;         // [M, K]
    const float *sA;          // [M, KB]
    const uint8_t *B;         // [N, K], or [E, N, K]
    const float *sB;          // [NB, KB], or [E, NB, KB]
    __nv_bfloat16 *C;         // [M, N]
    const int32_t *offsets;   // [E + 1] on the device, or null: one product over all rows
    uint32_t *status;
    int M, N, K, KB, E;
};

constexpr int ROWS_N = 16;   // rows of B per CTA

// Programmatic dependent launch: the next kernel of the stream may be set up while this
// one runs, and waits for this one's end (and its memory) before it reads or writes.
//
// So a kernel is live while the one before it still writes, and whatever that one may have
// written (a quantizer's codes and scales, a product's rows, any operand) is not read-only
// for the kernel's life: the kernels launched this way read global memory with ordinary
// loads, which the wait orders, and never through the non-coherent path.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void mma_e4m3_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16_if(const uint8_t *p, bool ok) {
    return ok ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0u, 0u, 0u, 0u);
}

// Rows of expert e: offsets clamped to [0, T]; a table that decreases or leaves
// [0, T] gives clamped ranges.
__device__ __forceinline__ void expert_rows(const int32_t *offsets, int e, int T, int &lo, int &hi) {
    lo = min(max(offsets[e], 0), T);
    hi = min(max(offsets[e + 1], 0), T);
}

// The `slot`-th expert that has rows (-1: there are fewer), found by the whole
// CTA; `found` is a shared word.  The CTAs of the last slot look at the whole
// table, and one of them reports a bad one.
__device__ __forceinline__ int busy_expert(const int32_t *offsets, int E, int T, int slot, int *counts, int *found,
                                           uint32_t *status) {
    const bool last = blockIdx.y + 1 == gridDim.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (threadIdx.x == 0) *found = -1;
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + static_cast<int>(threadIdx.x);
        int lo = 0, hi = 0;
        if (e < E) {
            expert_rows(offsets, e, T, lo, hi);
            if (last && blockIdx.x == 0 && (lo != offsets[e] || hi != offsets[e + 1] || hi < lo))
                atomicOr(status, STATUS_RECORD);
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, hi > lo);
        if (lane == 0) counts[warp] = __popc(mask);
        __syncthreads();
        int before = base;
        for (int w = 0; w < nw; ++w) {
            if (w == warp && hi > lo && before + __popc(mask & ((1u << lane) - 1u)) == slot) *found = e;
            before += counts[w];
        }
        base = before;
        __syncthreads();
        if (base > slot && !last) break;
    }
    return *found;
}

template <int NT, int U, int WARPS, int CTAS, bool NEXT>
__global__ void __launch_bounds__(WARPS * 32, CTAS) bsfp8_block128_rows(const RowsArgs a) {
    __shared__ float red[WARPS][NT][4][32];
    __shared__ int counts[WARPS];
    __shared__ int found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = static_cast<int>(blockIdx.x) * ROWS_N;
    wait_for_previous();
    int lo = 0, hi = a.M, e = 0;
    if (a.offsets) {
        e = busy_expert(a.offsets, a.E, a.M, static_cast<int>(blockIdx.y), counts, &found, a.status);
        if (e < 0) return;
        expert_rows(a.offsets, e, a.M, lo, hi);
    } else {
        lo = static_cast<int>(blockIdx.y) * 8 * NT;
        hi = min(hi, lo + 8 * NT);
    }
    const int NB = (a.N + 127) / 128;
    const uint8_t *B0 = a.B + (static_cast<int64_t>(e) * a.N + n0 + g) * a.K + 16 * t;
    const uint8_t *B1 = B0 + static_cast<int64_t>(8) * a.K;
    const bool ok1 = n0 + 8 < a.N;   // N is a multiple of 8: the rows n0 + g exist
    const float *sB = a.sB + (static_cast<int64_t>(e) * NB + n0 / 128) * a.KB;
    for (int m0 = lo; m0 < hi; m0 += 8 * NT) {
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][c] = 0.0f;
        for (int kb0 = warp; kb0 < a.KB; kb0 += WARPS * U) {
            uint4 w0[U][2], w1[U][2], x[U][NT][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = (kb0 + u * WARPS) * 128 + 64 * j;   // sizes are below 2^30: no overflow
                    const bool in = k + 16 * t < a.K;
                    w0[u][j] = load16_if(B0 + k, in);
                    w1[u][j] = load16_if(B1 + k, in && ok1);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int k = (kb0 + u * WARPS) * 128 + 64 * j + 16 * t;
                        const int m = m0 + 8 * n + g;
                        x[u][n][j] = load16_if(a.A + static_cast<int64_t>(m) * a.K + k, m < hi && k < a.K);
                    }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kb = kb0 + u * WARPS;
                if (kb < a.KB) {
                    const float sb = sB[kb];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            mma_e4m3_16x8x32(p, w0[u][j].x, w1[u][j].x, w0[u][j].y, w1[u][j].y, x[u][n][j].x, x[u][n][j].y);
                            mma_e4m3_16x8x32(p, w0[u][j].z, w1[u][j].z, w0[u][j].w, w1[u][j].w, x[u][n][j].z, x[u][n][j].w);
                        }
                        const int m = m0 + 8 * n + 2 * t;
                        const float *s = a.sA + static_cast<int64_t>(m) * a.KB + kb;
                        const float s0 = m < hi ? s[0] * sb : 0.0f;
                        const float s1 = m + 1 < hi ? s[a.KB] * sb : 0.0f;
                        acc[n][0] = fmaf(s0, p[0], acc[n][0]);
                        acc[n][1] = fmaf(s1, p[1], acc[n][1]);
                        acc[n][2] = fmaf(s0, p[2], acc[n][2]);
                        acc[n][3] = fmaf(s1, p[3], acc[n][3]);
                    }
                }
            }
        }
        if constexpr (NEXT) {
            if (m0 + 8 * NT >= hi) launch_dependents();
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) red[warp][n][c][lane] = acc[n][c];
        __syncthreads();
        // output i: row r of the 16, token j of the 8 NT
        for (int i = threadIdx.x; i < NT * 128; i += WARPS * 32) {
            const int r = i & 15, j = i >> 4, n = j >> 3, tok = j & 7;
            const int c = (r >> 3) * 2 + (tok & 1), l = (r & 7) * 4 + (tok >> 1);
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += red[w][n][c][l];
            if (m0 + j < hi && n0 + r < a.N)
                a.C[static_cast<int64_t>(m0 + j) * a.N + n0 + r] = __float2bfloat16_rn(v);
        }
        __syncthreads();
    }
}

}  // namespace bsfp8
