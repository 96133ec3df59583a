// moe_layer.cuh -- a whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   h[t,e] = silu(G_e x_t) * (U_e x_t)           gate and up rows of W1[e]
//   out[t] = bf16( sum over the token's experts w[t,e] * (D_e h[t,e]) )
//
// Weights are E4M3 codes with a scale for each 128 x 128 block; x is bf16 and is not
// quantized.  A few tokens leave the call bound by reading each busy expert's weights once
// (3 I H bytes), so the weights go from global memory straight to registers, as in the rows
// form of the products (block128_rows.cuh), and the arithmetic has to stay out of their way.
//
// Codes become fp16 by one conversion for two (every E4M3 value is an fp16 number), and
// x, h become fp16 with one power of two for a token's 128 (x) or 16 (h) values, which
// brings the largest of them to [2^14, 2^15): x keeps all its 8 bits down to 2^-28 of the
// largest, h 11 bits (half a step 2^-11, an eighth of the result's bf16 step).  The
// products of a 128-K block are summed in fp32 by mma.m16n8k16 (16 weight rows as its M
// side, 8 tokens as its N side), then acc += (scales) * sum in fp32.
//
// Each warp takes K blocks of its own and the warps' sums are added in warp order; which warp
// takes which block depends on the expert and the block alone, and experts are added in
// ascending order: calls repeat bit for bit, and a token's bits do not depend on the
// other tokens.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "block128_rows.cuh"

namespace bsfp8 {

constexpr int MOE_FEW_TOKENS = 8;   // the kernels of this file; more: moe_tile.cuh
constexpr int MOE_MAX_TOKENS = 64, MOE_MAX_TOP = 32, MOE_MAX_EXPERTS = 1024;
constexpr int MOE_WARPS = 8, MOE_THREADS = MOE_WARPS * 32;
constexpr int MOE_UP_COLS = 16;     // columns of h per CTA: 16 gate and 16 up rows
constexpr int MOE_DOWN_COLS = 32;   // columns of the output per CTA

struct MoeArgs {
    const __nv_bfloat16 *x;   // [T, H]
    const int32_t *ids;       // [T, top]; outside [0, E): no expert
    const float *w;           // [T, top]
    const uint8_t *W1, *W2;   // [E, 2I, H], [E, H, I]
    const float *s1, *s2;     // [E, ceil(2I/128), ceil(H/128)], [E, ceil(H/128), ceil(I/128)]
    __nv_bfloat16 *out;       // [T, H]
    __half *h;                // workspace: [T * top, I], and
    float *hs;                // [T * top, I / 16] powers of two: h times hs is the value
    int T, top, E, H, I;
};

__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ uint32_t half2_of_e4m3x2_hi(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ void mma_f16_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_rn(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The power of two that brings amax to [2^14, 2^15), and its inverse.  Below 2^-112 the
// same one is taken (the values get subnormal steps of 2^-136 then).
__device__ __forceinline__ float scale_to_half(float amax, float &inverse) {
    const uint32_t e = max(__float_as_uint(amax) >> 23, 15u);
    inverse = __uint_as_float((e - 14u) << 23);
    return __uint_as_float((268u - e) << 23);
}

// A lane's 32 values of a token's 128-K block (the quad holds all of them) as fp16; returns
// the inverse of their scale.
__device__ __forceinline__ float block_to_half(const uint4 (&x)[4], uint32_t (&r)[16]) {
    uint32_t w[16], m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * i] = x[i].x, w[4 * i + 1] = x[i].y, w[4 * i + 2] = x[i].z, w[4 * i + 3] = x[i].w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint32_t v;
        asm("abs.bf16x2 %0, %1;" : "=r"(v) : "r"(w[i]));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(v));
    }
    float amax = fmaxf(bf16_lo(m), bf16_hi(m));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    float inverse;
    const float s = scale_to_half(amax, inverse);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = half2_rn(bf16_lo(w[i]) * s, bf16_hi(w[i]) * s);
    return inverse;
}

// The sums of two 16-row pieces (a, b: row g, row g + 8 of each) of a weight's 128-K block
// with N groups of eight tokens.
template <int N>
__device__ __forceinline__ void block_products(float (&p)[N][2][4], const uint4 (&a)[2][2], const uint4 (&b)[2][2],
                                               const uint32_t (&x)[N][16]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) p[n][i][c] = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t wa[4] = {a[i][j].x, a[i][j].y, a[i][j].z, a[i][j].w};
            const uint32_t wb[4] = {b[i][j].x, b[i][j].y, b[i][j].z, b[i][j].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t a0 = half2_of_e4m3x2(wa[c]), a1 = half2_of_e4m3x2(wb[c]);
                const uint32_t a2 = half2_of_e4m3x2_hi(wa[c]), a3 = half2_of_e4m3x2_hi(wb[c]);
#pragma unroll
                for (int n = 0; n < N; ++n)
                    mma_f16_16x8x16(p[n][i], a0, a1, a2, a3, x[n][8 * j + 2 * c], x[n][8 * j + 2 * c + 1]);
            }
        }
}

// Whether pair p = (t, j) is the first of its token with this expert (the later ones only
// add their weight to it).
__device__ __forceinline__ bool first_of_token(const MoeArgs &a, int p, int e) {
    for (int q = p - p % a.top; q < p; ++q)
        if (a.ids[q] == e) return false;
    return true;
}

// silu(g) * u.  Deep in the negative gates the exponential's two halves go to one factor
// each, so that a large u brings back what the exponential alone would lose.
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float t = g * 1.44269504f;
    float n;   // 2^(-|t| / 2), subnormal numbers included
    asm("ex2.approx.f32 %0, %1;" : "=f"(n) : "f"(-0.5f * fabsf(t)));
    const float r = rcp(fmaf(n, n, 1.0f));
    return t < 0.0f ? (g * n) * (u * n) * r : (g * r) * u;
}

// Gate and up: a CTA owns 16 columns of h of one busy expert, and all of its tokens, eight
// times NT at a time.  MMA piece i holds gate rows 8 i .. 8 i + 7 and the up rows of the same
// columns, so that a thread has both numbers of an h.
template <int NT>
__global__ void __launch_bounds__(MOE_THREADS, NT == 1 ? 2 : 1) bsfp8_moe_up(const MoeArgs a) {
    __shared__ uint32_t bits[MOE_MAX_EXPERTS / 32];
    __shared__ int found, count;
    __shared__ uint16_t list[MOE_MAX_TOKENS];   // pairs: one for each of the expert's tokens
    __shared__ float red[MOE_WARPS][NT][2][4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int pairs = a.T * a.top, n0 = static_cast<int>(blockIdx.x) * MOE_UP_COLS;
    if (threadIdx.x < MOE_MAX_EXPERTS / 32) bits[threadIdx.x] = 0u;
    if (threadIdx.x == 0) found = -1, count = 0;
    __syncthreads();
    wait_for_previous();
    for (int p = threadIdx.x; p < pairs; p += MOE_THREADS) {
        const uint32_t e = static_cast<uint32_t>(a.ids[p]);
        if (e < static_cast<uint32_t>(a.E)) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (warp == 0) {   // the blockIdx.y-th busy expert
        const uint32_t b = bits[lane];
        int sum = __popc(b);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        const int k = static_cast<int>(blockIdx.y) - (sum - __popc(b));
        if (k >= 0 && k < __popc(b)) {
            uint32_t left = b;
            for (int i = 0; i < k; ++i) left &= left - 1u;
            found = 32 * lane + __ffs(left) - 1;
        }
    }
    __syncthreads();
    const int e = found;
    if (e < 0) return;
    for (int p = threadIdx.x; p < pairs; p += MOE_THREADS)
        if (a.ids[p] == e && first_of_token(a, p, e)) list[atomicAdd(&count, 1)] = static_cast<uint16_t>(p);
    __syncthreads();
    const int n = count, KB = (a.H + 127) / 128, NB = (2 * a.I + 127) / 128;
    const uint8_t *W = a.W1 + (static_cast<int64_t>(e) * 2 * a.I + n0 + g) * a.H + 16 * t;
    const int64_t up = static_cast<int64_t>(a.I) * a.H, eight = static_cast<int64_t>(8) * a.H;
    const float *sg = a.s1 + (static_cast<int64_t>(e) * NB + n0 / 128) * KB;
    const float *su = a.s1 + (static_cast<int64_t>(e) * NB + (a.I + n0) / 128) * KB;
    for (int m0 = 0; m0 < n; m0 += 8 * NT) {
        float acc[NT][2][4];
        const __nv_bfloat16 *x[NT];
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const int m = m0 + 8 * k + g;
            x[k] = m < n ? a.x + static_cast<int64_t>(list[m] / a.top) * a.H + 16 * t : nullptr;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[k][i][c] = 0.0f;
        }
        for (int kb = warp; kb < KB; kb += MOE_WARPS) {
            uint4 wg[2][2], wu[2][2], xr[NT][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = kb * 128 + 64 * j;
                const bool in = k + 16 * t < a.H;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    wg[i][j] = load16_if(W + i * eight + k, in);
                    wu[i][j] = load16_if(W + up + i * eight + k, in);
                }
#pragma unroll
                for (int m = 0; m < NT; ++m)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        xr[m][2 * j + c] = load16_if(reinterpret_cast<const uint8_t *>(x[m] + k + 8 * c), in && x[m]);
            }
            const float s_gate = sg[kb], s_up = su[kb];
            uint32_t xh[NT][16];
            float inverse[NT], p[NT][2][4];
#pragma unroll
            for (int m = 0; m < NT; ++m) inverse[m] = block_to_half(xr[m], xh[m]);
            block_products<NT>(p, wg, wu, xh);
#pragma unroll
            for (int m = 0; m < NT; ++m) {   // columns 2 t and 2 t + 1: the tokens of lanes 8 t and 8 t + 4
                const float i0 = __shfl_sync(0xFFFFFFFFu, inverse[m], 8 * t);
                const float i1 = __shfl_sync(0xFFFFFFFFu, inverse[m], 8 * t + 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    acc[m][i][0] = fmaf(s_gate * i0, p[m][i][0], acc[m][i][0]);
                    acc[m][i][1] = fmaf(s_gate * i1, p[m][i][1], acc[m][i][1]);
                    acc[m][i][2] = fmaf(s_up * i0, p[m][i][2], acc[m][i][2]);
                    acc[m][i][3] = fmaf(s_up * i1, p[m][i][3], acc[m][i][3]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) red[warp][k][i][c][lane] = acc[k][i][c];
        __syncthreads();
        // sixteen threads have a token's columns
        for (int i = threadIdx.x; i < NT * 128; i += MOE_THREADS) {
            const int col = i & 15, m = i >> 4, k = m >> 3, tok = m & 7;
            const int piece = col >> 3, c = tok & 1, l = (col & 7) * 4 + (tok >> 1);
            float gate = 0.0f, upv = 0.0f;
#pragma unroll
            for (int w = 0; w < MOE_WARPS; ++w) {
                gate += red[w][k][piece][c][l];
                upv += red[w][k][piece][2 + c][l];
            }
            const float v = silu_mul(gate, upv);
            float amax = fabsf(v);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            float inverse;
            const float s = scale_to_half(amax, inverse);
            if (m0 + m < n) {
                const int64_t pair = list[m0 + m];
                a.h[pair * a.I + n0 + col] = __float2half_rn(v * s);
                if (col == 0) a.hs[pair * (a.I / 16) + n0 / 16] = inverse;
            }
        }
        __syncthreads();
    }
    launch_dependents();
}

// The experts' tokens, in shared memory: one entry for each token of an expert, from start[e]
// to start[e + 1].
struct MoeLists {
    int *start;          // [E + 1]
    int *experts;        // how many are busy, and the most tokens of one
    uint16_t *busy;      // [E] which, ascending
    uint16_t *pair;      // [pairs] the row of h: the token's first pair with the expert
    uint16_t *token;     // [pairs]
    float *weight;       // [pairs] the sum of the token's weights for the expert
    uint16_t *id;        // [pairs] while the lists are made: the pairs' experts,
    uint8_t *number;     // [pairs] and their numbers among the expert's
};

__host__ __device__ constexpr int moe_pad16(int v) { return (v + 15) / 16 * 16; }

struct MoeListsLayout {
    int start, busy, pair, token, weight, id, number, bytes;   // offsets
};

__host__ __device__ inline MoeListsLayout moe_lists_layout(int T, int top, int E) {
    MoeListsLayout s{};
    s.start = 16;   // the number of busy experts is before it
    s.busy = s.start + moe_pad16(4 * (E + 1));
    s.pair = s.busy + moe_pad16(2 * E);
    s.token = s.pair + moe_pad16(2 * T * top);
    s.weight = s.token + moe_pad16(2 * T * top);
    s.id = s.weight + moe_pad16(4 * T * top);
    s.number = s.id + moe_pad16(2 * T * top);
    s.bytes = s.number + moe_pad16(T * top);
    return s;
}

__device__ __forceinline__ MoeLists moe_lists(uint8_t *at, int T, int top, int E) {
    const MoeListsLayout o = moe_lists_layout(T, top, E);
    MoeLists l;
    l.experts = reinterpret_cast<int *>(at);
    l.start = reinterpret_cast<int *>(at + o.start);
    l.busy = reinterpret_cast<uint16_t *>(at + o.busy);
    l.pair = reinterpret_cast<uint16_t *>(at + o.pair);
    l.token = reinterpret_cast<uint16_t *>(at + o.token);
    l.weight = reinterpret_cast<float *>(at + o.weight);
    l.id = reinterpret_cast<uint16_t *>(at + o.id);
    l.number = at + o.number;
    return l;
}

// Made by the whole CTA: the ids come to shared memory, each pair that is its token's first
// with the expert takes a number there, and the ranges follow from how many there are (the
// order in a range does not matter: each entry is a column of its own).
__device__ __forceinline__ void build_lists(const MoeArgs &a, const MoeLists &l) {
    const int lane = threadIdx.x & 31, threads = blockDim.x, pairs = a.T * a.top;
    constexpr uint16_t NONE = 0xFFFF;
    for (int i = threadIdx.x; i <= a.E; i += threads) l.start[i] = 0;
    for (int p = threadIdx.x; p < pairs; p += threads) {
        const uint32_t e = static_cast<uint32_t>(a.ids[p]);
        l.id[p] = e < static_cast<uint32_t>(a.E) ? static_cast<uint16_t>(e) : NONE;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += threads) {
        const uint16_t e = l.id[p];
        bool first = e != NONE;
        for (int q = p - p % a.top; q < p; ++q) first &= l.id[q] != e;
        l.number[p] = first ? static_cast<uint8_t>(atomicAdd(&l.start[e], 1)) : 255;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int base = 0, used = 0, most = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, c = e < a.E ? l.start[e] : 0;
            most = max(most, c);
            int sum = c;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, k);
                if (lane >= k) sum += v;
            }
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, c > 0);
            if (e < a.E) l.start[e] = base + sum - c;
            if (c > 0) l.busy[used + __popc(mask & ((1u << lane) - 1u))] = static_cast<uint16_t>(e);
            base += __shfl_sync(0xFFFFFFFFu, sum, 31);
            used += __popc(mask);
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (lane == 0) {
            l.experts[0] = used;
            l.experts[1] = most;
            l.start[a.E] = base;
        }
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += threads) {
        if (l.number[p] == 255) continue;
        const int e = l.id[p], t = p / a.top, at = l.start[e] + l.number[p];
        float w = a.w[p];
        for (int q = p + 1; q < (t + 1) * a.top; ++q)
            if (l.id[q] == e) w += a.w[q];
        l.pair[at] = static_cast<uint16_t>(p);
        l.token[at] = static_cast<uint16_t>(t);
        l.weight[at] = w;
    }
    __syncthreads();
}

// Shared memory of the down kernel: the lists, and sums [warps][T][columns + 8].
__host__ __device__ inline int moe_down_shared(int T, int top, int E) {
    return moe_lists_layout(T, top, E).bytes + 4 * MOE_WARPS * T * (MOE_DOWN_COLS + 8);
}

// Down and the weighted sum: a CTA owns 32 columns of the output for all tokens and
// passes over the busy experts in ascending order.  Each warp adds what its K blocks give
// to sums of its own in shared memory.
__global__ void __launch_bounds__(MOE_THREADS, 2) bsfp8_moe_down(const MoeArgs a) {
    extern __shared__ __align__(16) uint8_t moe_smem[];
    const MoeLists L = moe_lists(moe_smem, a.T, a.top, a.E);
    float *sums = reinterpret_cast<float *>(moe_smem + moe_lists_layout(a.T, a.top, a.E).bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = static_cast<int>(blockIdx.x) * MOE_DOWN_COLS;
    constexpr int LD = MOE_DOWN_COLS + 8;
    for (int i = threadIdx.x; i < MOE_WARPS * a.T * LD; i += MOE_THREADS) sums[i] = 0.0f;
    wait_for_previous();
    build_lists(a, L);
    const int KB = (a.I + 127) / 128, NB = (a.H + 127) / 128, chunks = a.I / 16;
    const bool second = n0 + 16 < a.H;   // H is a multiple of 16
    float *mine = sums + warp * a.T * LD;
    for (int b = 0; b < *L.experts; ++b) {
        const int e = L.busy[b], first = L.start[e], n = L.start[e + 1] - first;
        const uint8_t *W = a.W2 + (static_cast<int64_t>(e) * a.H + n0 + g) * a.I + 16 * t;
        const float *s2 = a.s2 + (static_cast<int64_t>(e) * NB + n0 / 128) * KB;
        // K block kb of expert e belongs to warp (e KB + kb) mod warps
        for (int kb = (warp + MOE_WARPS - (e % MOE_WARPS) * (KB % MOE_WARPS) % MOE_WARPS) % MOE_WARPS; kb < KB; kb += MOE_WARPS) {
            uint4 wa[2][2], wb[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = kb * 128 + 64 * j;
                const bool in = k + 16 * t < a.I;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    wa[i][j] = load16_if(W + static_cast<int64_t>(16 * i) * a.I + k, in && (i == 0 || second));
                    wb[i][j] = load16_if(W + static_cast<int64_t>(16 * i + 8) * a.I + k, in && (i == 0 || second));
                }
            }
            const float sb = s2[kb];
            for (int m0 = 0; m0 < n; m0 += 8) {
                uint32_t xh[1][16];
                float sc[2];
                const int64_t pair = m0 + g < n ? L.pair[first + m0 + g] : -1;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = kb * 128 + 64 * j + 16 * t;
                    const bool in = pair >= 0 && k < a.I;
                    const uint8_t *h = reinterpret_cast<const uint8_t *>(a.h + pair * a.I + k);
                    sc[j] = in ? a.hs[pair * chunks + k / 16] : 0.0f;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 v = load16_if(h + 16 * c, in);
                        xh[0][8 * j + 4 * c] = v.x, xh[0][8 * j + 4 * c + 1] = v.y;
                        xh[0][8 * j + 4 * c + 2] = v.z, xh[0][8 * j + 4 * c + 3] = v.w;
                    }
                }
                // one scale for the block: the largest of its eight
                float most = fmaxf(fmaxf(sc[0], sc[1]), 0x1p-126f);
                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                const float r = __uint_as_float((254u << 23) - __float_as_uint(most));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const __half2 f = __float2half2_rn(sc[j] * r);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&xh[0][8 * j + c]), f);
                        xh[0][8 * j + c] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                }
                float p[1][2][4];
                block_products<1>(p, wa, wb, xh);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float s = sb * __shfl_sync(0xFFFFFFFFu, most, 8 * t + 4 * c);
                    const int m = m0 + 2 * t + c;
                    if (m < n) {
                        const float f = s * L.weight[first + m];
                        float *to = mine + L.token[first + m] * LD + g;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            to[16 * i] = fmaf(f, p[0][i][c], to[16 * i]);
                            to[16 * i + 8] = fmaf(f, p[0][i][2 + c], to[16 * i + 8]);
                        }
                    }
                }
                __syncwarp();
            }
        }
    }
    launch_dependents();
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * MOE_DOWN_COLS; i += MOE_THREADS) {
        const int tok = i / MOE_DOWN_COLS, c = i % MOE_DOWN_COLS;
        if (n0 + c >= a.H) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < MOE_WARPS; ++w) v += sums[(w * a.T + tok) * LD + c];
        a.out[static_cast<int64_t>(tok) * a.H + n0 + c] = __float2bfloat16_rn(v);
    }
}

}  // namespace bsfp8
