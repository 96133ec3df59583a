// moe_layer.cuh -- a whole mixture-of-experts layer for a few tokens, eight at a time, in two
// kernels.
//
//   h[t,e] = silu(G_e x_t) * (U_e x_t)           gate and up rows of W1[e]
//   out[t] = bf16( sum over the token's experts w[t,e] * (D_e h[t,e]) )
//
// Weights are E4M3 codes with a scale for each 128 x 128 block; x is bf16 and is not
// quantized.  A few tokens leave the call bound by reading each busy expert's weights once
// (3 I H bytes), so what counts is how many bytes are on their way: each thread copies the
// 16-byte pieces that it will multiply to shared memory of its own, some K blocks ahead, and
// takes them from there without a barrier (3 tokens, 8 of 64 experts of 7168 x 2048, 16 of them
// busy: 120 us, 5.9 TB/s; held in registers, one block ahead, 143).  1 token, 4 of 32 of 2048 x
// 1024: 11.0 us, 25 MB (8.8 with the weights in L2); there the two launches and the first loads of
// each are most of it.
//
// More than eight tokens are as many calls side by side (the grid's z), which share the weights in
// L2: with small weights that costs less than the set-up of moe_tile.cuh (the rule of moe_api.cu).
//
// Two launches and not one: the down product needs all of h, and no CTA waits for another.
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
// ascending order: calls repeat bit for bit, and within these kernels a token's bits do not
// depend on the other tokens.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "block128_rows.cuh"

namespace bsfp8 {

constexpr int MOE_FEW_TOKENS = 8;   // tokens of a CTA of this file: the MMA's columns
constexpr int MOE_MAX_TOKENS = 64, MOE_MAX_TOP = 32, MOE_MAX_EXPERTS = 1024;
constexpr int MOE_UP_WARPS = 8, MOE_DOWN_WARPS = 16;
constexpr int MOE_UP_COLS = 16;     // columns of h per CTA: 16 gate and 16 up rows

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

// The power of two that brings amax to [2^TOP, 2^(TOP + 1)), and its inverse.  Below 2^(TOP - 126)
// the same one is taken (14: the values get subnormal steps of 2^-136 then).
template <int TOP = 14>
__device__ __forceinline__ float scale_to_half(float amax, float &inverse) {
    const uint32_t e = max(__float_as_uint(amax) >> 23, TOP + 1u);
    inverse = __uint_as_float((e - TOP) << 23);
    return __uint_as_float((254u + TOP - e) << 23);
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

// The sums of a 16-row piece (a: row g, b: row g + 8) of a weight's 128-K block with eight tokens.
__device__ __forceinline__ void block_product(float (&p)[4], const uint4 (&a)[2], const uint4 (&b)[2],
                                              const uint32_t (&x)[16]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) p[c] = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t wa[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
        const uint32_t wb[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
            mma_f16_16x8x16(p, half2_of_e4m3x2(wa[c]), half2_of_e4m3x2(wb[c]), half2_of_e4m3x2_hi(wa[c]),
                            half2_of_e4m3x2_hi(wb[c]), x[8 * j + 2 * c], x[8 * j + 2 * c + 1]);
    }
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

// Up to eight tokens are the columns of every MMA, whichever of them an expert has.  An expert's
// tokens as a warp sees them: bit p of the mask is pair p = (token, j), 32 PW pairs at most.
template <int PW>
struct MoePairs {
    uint32_t bits[PW];   // the same in every lane
    // The token's pairs with the expert, bit j for pair (token, j).
    __device__ __forceinline__ uint32_t of(int token, int top) const {
        const int at = token * top;
        uint32_t lo = 0u, hi = 0u;
#pragma unroll
        for (int i = 0; i < PW; ++i) {
            if (i == at >> 5) lo = bits[i];
            if (i == (at >> 5) + 1) hi = bits[i];
        }
        return __funnelshift_r(lo, hi, at & 31) & (top == 32 ? 0xFFFFFFFFu : (1u << top) - 1u);
    }
    // The first of them, or -1.
    __device__ __forceinline__ int first(int token, int top) const {
        const uint32_t w = of(token, top);
        return w ? token * top + __ffs(w) - 1 : -1;
    }
};

// Pairs with expert e; own: the lane's ids (pair 32 i + lane), -1 past the end.
template <int PW>
__device__ __forceinline__ MoePairs<PW> pairs_of(const int (&own)[PW], int e) {
    MoePairs<PW> m;
#pragma unroll
    for (int i = 0; i < PW; ++i) m.bits[i] = __ballot_sync(0xFFFFFFFFu, own[i] == e);
    return m;
}

// Ids of the pairs p0 .. p0 + pairs - 1.
template <int PW>
__device__ __forceinline__ void load_ids(const MoeArgs &a, int p0, int pairs, int (&own)[PW]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < PW; ++i) own[i] = 32 * i + lane < pairs ? a.ids[p0 + 32 * i + lane] : -1;
}

// A thread's 16-byte pieces of a K block in shared memory: N of them, DEPTH blocks.
template <int N, int DEPTH>
struct MoeRing {
    uint8_t *mine;
    __device__ __forceinline__ explicit MoeRing(uint8_t *smem)
        : mine(smem + (threadIdx.x >> 5) * (N * DEPTH * 512) + (threadIdx.x & 31) * 16) {}
    // Zeros where there is nothing to copy.
    __device__ __forceinline__ void copy(int slot, int i, const uint8_t *from, bool in) const {
        cp_async_16(smem_u32(mine + (slot * N + i) * 512), from, in ? 16u : 0u);
    }
    __device__ __forceinline__ uint4 get(int slot, int i) const {
        return *reinterpret_cast<const uint4 *>(mine + (slot * N + i) * 512);
    }
};

// Gate and up: a CTA owns 16 columns of h of one expert, for all of its tokens among eight.  The
// CTAs of pair blockIdx.y do this where it is the first of all with its expert, and leave otherwise.
// MMA piece i holds gate rows 8 i .. 8 i + 7 and the up rows of the same columns, so that a
// thread has both numbers of an h.
constexpr int MOE_UP_DEPTH = 3;
constexpr int MOE_UP_SMEM = MOE_UP_WARPS * MOE_UP_DEPTH * 8 * 512;

template <int PW>
__global__ void __launch_bounds__(MOE_UP_WARPS * 32, 2) bsfp8_moe_up(const MoeArgs a) {
    extern __shared__ __align__(16) uint8_t moe_smem[];
    __shared__ float red[MOE_UP_WARPS][2][4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = static_cast<int>(blockIdx.x) * MOE_UP_COLS;
    const MoeRing<8, MOE_UP_DEPTH> ring(moe_smem);
    wait_for_previous();
    const int t0 = static_cast<int>(blockIdx.z) * MOE_FEW_TOKENS, p0 = t0 * a.top;
    const int pairs = min(MOE_FEW_TOKENS, a.T - t0) * a.top;
    if (static_cast<int>(blockIdx.y) >= pairs) return;   // the last eight may be fewer
    int own[PW];
    load_ids<PW>(a, p0, pairs, own);
    const int e = a.ids[p0 + blockIdx.y];
    if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(a.E)) return;
    const int KB = (a.H + 127) / 128, NB = (2 * a.I + 127) / 128;
    const uint8_t *W = a.W1 + (static_cast<int64_t>(e) * 2 * a.I + n0 + g) * a.H + 16 * t;
    const int64_t up = static_cast<int64_t>(a.I) * a.H, eight = static_cast<int64_t>(8) * a.H;
    auto fetch = [&](int slot, int kb) {
        if (kb < KB) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = kb * 128 + 64 * j;
                const bool in = k + 16 * t < a.H;
                const uint8_t *from = in ? W + k : W;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ring.copy(slot, 4 * j + 2 * i, from + i * eight, in);
                    ring.copy(slot, 4 * j + 2 * i + 1, from + up + i * eight, in);
                }
            }
        }
        cp_async_commit();
    };
    const MoePairs<PW> m = pairs_of<PW>(own, e);
    {   // an earlier pair has this expert: its CTAs do the work
        bool earlier = false;
#pragma unroll
        for (int i = 0; i < PW; ++i) {
            const int left = static_cast<int>(blockIdx.y) - 32 * i;
            earlier |= left > 0 && (m.bits[i] & (left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u)) != 0u;
        }
        if (earlier) return;
    }
#pragma unroll
    for (int d = 0; d < MOE_UP_DEPTH; ++d) fetch(d, warp + d * MOE_UP_WARPS);
    const bool has = m.first(g, a.top) >= 0;   // this lane's token (none from T on)
    const __nv_bfloat16 *x = a.x + (has ? static_cast<int64_t>(t0 + g) * a.H + 16 * t : 0);
    const float *sg = a.s1 + (static_cast<int64_t>(e) * NB + n0 / 128) * KB;
    const float *su = a.s1 + (static_cast<int64_t>(e) * NB + (a.I + n0) / 128) * KB;
    uint4 xr[4];
    float s_gate = 0.0f, s_up = 0.0f;
    auto load_x = [&](int kb) {   // and the block's scales
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int k = kb * 128 + 64 * (c >> 1);
            xr[c] = load16_if(reinterpret_cast<const uint8_t *>(x + k + 8 * (c & 1)), has && k + 16 * t < a.H);
        }
        s_gate = sg[kb];
        s_up = su[kb];
    };
    if (warp < KB) load_x(warp);
    float acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
    int slot = 0;
    for (int kb = warp; kb < KB; kb += MOE_UP_WARPS) {
        uint32_t xh[16];
        const float inverse = block_to_half(xr, xh), gate = s_gate, upward = s_up;
        if (kb + MOE_UP_WARPS < KB) load_x(kb + MOE_UP_WARPS);
        // columns 2 t and 2 t + 1: the tokens of lanes 8 t and 8 t + 4
        const float i0 = __shfl_sync(0xFFFFFFFFu, inverse, 8 * t), i1 = __shfl_sync(0xFFFFFFFFu, inverse, 8 * t + 4);
        cp_async_wait_group<MOE_UP_DEPTH - 1>();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint4 wg[2], wu[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) wg[j] = ring.get(slot, 4 * j + 2 * i), wu[j] = ring.get(slot, 4 * j + 2 * i + 1);
            float p[4];
            block_product(p, wg, wu, xh);
            acc[i][0] = fmaf(gate * i0, p[0], acc[i][0]);
            acc[i][1] = fmaf(gate * i1, p[1], acc[i][1]);
            acc[i][2] = fmaf(upward * i0, p[2], acc[i][2]);
            acc[i][3] = fmaf(upward * i1, p[3], acc[i][3]);
        }
        fetch(slot, kb + MOE_UP_DEPTH * MOE_UP_WARPS);
        slot = slot + 1 == MOE_UP_DEPTH ? 0 : slot + 1;
    }
    launch_dependents();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) red[warp][i][c][lane] = acc[i][c];
    __syncthreads();
    // sixteen threads have a token's columns
    if (threadIdx.x < 128) {
        const int col = lane & 15, tok = static_cast<int>(threadIdx.x) >> 4;
        const int piece = col >> 3, c = tok & 1, l = (col & 7) * 4 + (tok >> 1);
        float gate = 0.0f, upv = 0.0f;
#pragma unroll
        for (int w = 0; w < MOE_UP_WARPS; ++w) {
            gate += red[w][piece][c][l];
            upv += red[w][piece][2 + c][l];
        }
        const float v = silu_mul(gate, upv);
        float amax = fabsf(v);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        float inverse;
        const float s = scale_to_half(amax, inverse);
        const int first = m.first(tok, a.top);
        if (first >= 0) {
            const int64_t to = p0 + first;
            a.h[to * a.I + n0 + col] = __float2half_rn(v * s);
            if (col == 0) a.hs[to * (a.I / 16) + n0 / 16] = inverse;
        }
    }
}

// Down and the weighted sum: a CTA owns 16 MT columns of the output for eight tokens and passes
// over the busy experts in ascending order, DEPTH of a warp's blocks on their way.  Their weights
// and the routing are not written by the up kernel, and what came before that had ended when
// it let this kernel start: only h waits for it.
__host__ __device__ constexpr int moe_down_depth(int MT) { return MT == 1 ? 4 : MT == 2 ? 3 : 2; }
__host__ __device__ constexpr int moe_down_smem(int MT) { return MOE_DOWN_WARPS * moe_down_depth(MT) * 4 * MT * 512; }

template <int MT, int PW>
__global__ void __launch_bounds__(MOE_DOWN_WARPS * 32, 1) bsfp8_moe_down(const MoeArgs a) {
    constexpr int DEPTH = moe_down_depth(MT);
    extern __shared__ __align__(16) uint8_t moe_smem[];
    __shared__ uint32_t bits[MOE_MAX_EXPERTS / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = static_cast<int>(blockIdx.x) * 16 * MT;
    const MoeRing<4 * MT, DEPTH> ring(moe_smem);
    const int t0 = static_cast<int>(blockIdx.z) * MOE_FEW_TOKENS, p0 = t0 * a.top, tokens = min(MOE_FEW_TOKENS, a.T - t0);
    int own[PW];
    load_ids<PW>(a, p0, tokens * a.top, own);
    if (threadIdx.x < MOE_MAX_EXPERTS / 32) bits[threadIdx.x] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PW; ++i)
        if (i == warp && static_cast<uint32_t>(own[i]) < static_cast<uint32_t>(a.E))
            atomicOr(&bits[own[i] >> 5], 1u << (own[i] & 31));
    __syncthreads();
    const int KB = (a.I + 127) / 128, NB = (a.H + 127) / 128, chunks = a.I / 16;
    uint32_t left = bits[lane];   // experts of 32 lane .. that are still to come
    // K block kb of expert e belongs to warp (e KB + kb) mod warps; the warp's next one
    int e = -1, kb = KB;
    auto next = [&]() {
        kb += MOE_DOWN_WARPS;
        while (kb >= KB) {
            const uint32_t any = __ballot_sync(0xFFFFFFFFu, left != 0u);
            if (!any) return false;
            const int src = __ffs(any) - 1;
            const uint32_t word = __shfl_sync(0xFFFFFFFFu, left, src);
            e = 32 * src + __ffs(word) - 1;
            if (lane == src) left &= left - 1u;
            kb = (warp + MOE_DOWN_WARPS - (e % MOE_DOWN_WARPS) * (KB % MOE_DOWN_WARPS) % MOE_DOWN_WARPS) % MOE_DOWN_WARPS;
        }
        return true;
    };
    int es[DEPTH], ks[DEPTH];   // the blocks on their way (-1: none)
    auto fetch = [&](int u) {
        es[u] = next() ? e : -1;
        ks[u] = kb;
        if (es[u] >= 0) {
            const uint8_t *W = a.W2 + (static_cast<int64_t>(e) * a.H + n0 + g) * a.I + 16 * t;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = kb * 128 + 64 * j;
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {   // eight rows each
                    const bool in = k + 16 * t < a.I && n0 + 8 * i < a.H;
                    ring.copy(u, 2 * i + j, in ? W + static_cast<int64_t>(8 * i) * a.I + k : a.W2, in);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) fetch(u);
    uint4 hr[4];
    float sc[2], w = 0.0f, sb[MT];
    bool has = false;
    auto load_h = [&](int u) {   // a token's values, their scales, its weight and the block's scales
        if (es[u] < 0) return;
        const uint32_t mine = pairs_of<PW>(own, es[u]).of(g, a.top);   // none from T on
        has = mine != 0u;
        const int64_t pair = has ? p0 + g * a.top + __ffs(mine) - 1 : 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = ks[u] * 128 + 64 * j + 16 * t;
            const bool in = has && k < a.I;
            const uint8_t *h = reinterpret_cast<const uint8_t *>(a.h + pair * a.I + (in ? k : 0));
            sc[j] = in ? a.hs[pair * chunks + k / 16] : 0.0f;
            hr[2 * j] = load16_if(h, in);
            hr[2 * j + 1] = load16_if(h + 16, in);
        }
        w = has ? a.w[pair] : 0.0f;   // and its other weights for the expert
        for (uint32_t rest = mine & (mine - 1u); rest; rest &= rest - 1u) w += a.w[p0 + g * a.top + __ffs(rest) - 1];
#pragma unroll
        for (int i = 0; i < MT; ++i)
            sb[i] = a.s2[(static_cast<int64_t>(es[u]) * NB + min((n0 + 16 * i) / 128, NB - 1)) * KB + ks[u]];
    };
    wait_for_previous();
    load_h(0);
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
    while (es[0] >= 0) {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            if (es[u] < 0) break;
            // one scale for the block: the largest of its eight
            float most = fmaxf(fmaxf(sc[0], sc[1]), 0x1p-126f);
            most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
            const float r = __uint_as_float((254u << 23) - __float_as_uint(most));
            uint32_t xh[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const __half2 f = __float2half2_rn(sc[j] * r);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t v[4] = {hr[2 * j + c].x, hr[2 * j + c].y, hr[2 * j + c].z, hr[2 * j + c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&v[k]), f);
                        xh[8 * j + 4 * c + k] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                }
            }
            float wt[2], f[2], s[MT];
            bool hs[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                wt[c] = __shfl_sync(0xFFFFFFFFu, w, 8 * t + 4 * c);
                f[c] = __shfl_sync(0xFFFFFFFFu, most, 8 * t + 4 * c);
                hs[c] = __shfl_sync(0xFFFFFFFFu, has, 8 * t + 4 * c);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) s[i] = sb[i];
            load_h((u + 1) % DEPTH);
            cp_async_wait_group<DEPTH - 1>();
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint4 wa[2], wb[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) wa[j] = ring.get(u, 4 * i + j), wb[j] = ring.get(u, 4 * i + 2 + j);
                float p[4];
                block_product(p, wa, wb, xh);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (hs[c]) {   // (a token without the expert has nothing here, not zero times something)
                        acc[i][c] = fmaf(wt[c], s[i] * f[c] * p[c], acc[i][c]);
                        acc[i][2 + c] = fmaf(wt[c], s[i] * f[c] * p[2 + c], acc[i][2 + c]);
                    }
            }
            fetch(u);
        }
    }
    launch_dependents();
    cp_async_wait_all();
    __syncthreads();   // the ring's memory is free
    float *red = reinterpret_cast<float *>(moe_smem);   // [warps][MT][4][32]
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) red[((warp * MT + i) * 4 + c) * 32 + lane] = acc[i][c];
    __syncthreads();
    for (int o = threadIdx.x; o < 8 * 16 * MT; o += MOE_DOWN_WARPS * 32) {
        const int col = o % (16 * MT), tok = o / (16 * MT);
        const int c = (col >> 3 & 1) * 2 + (tok & 1), l = (col & 7) * 4 + (tok >> 1);
        float v = 0.0f;
#pragma unroll
        for (int x = 0; x < MOE_DOWN_WARPS; ++x) v += red[((x * MT + (col >> 4)) * 4 + c) * 32 + l];
        if (tok < tokens && n0 + col < a.H) a.out[static_cast<int64_t>(t0 + tok) * a.H + n0 + col] = __float2bfloat16_rn(v);
    }
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
    uint8_t *number;     // [pairs] and their numbers among the expert's,
    int *count;          // [E] which has so many
};

__host__ __device__ constexpr int moe_pad16(int v) { return (v + 15) / 16 * 16; }

struct MoeListsLayout {
    int start, busy, pair, token, weight, id, number, count, bytes;   // offsets
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
    s.count = s.number + moe_pad16(T * top);
    s.bytes = s.count + moe_pad16(4 * E);
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
    l.count = reinterpret_cast<int *>(at + o.count);
    return l;
}

// Made by the whole CTA: the ids come to shared memory, each pair that is its token's first
// with the expert takes a number there, and the ranges follow from how many there are (the
// order in a range does not matter: each entry is a column of its own).
__device__ __forceinline__ void build_lists(const MoeArgs &a, const MoeLists &l) {
    const int lane = threadIdx.x & 31, threads = blockDim.x, pairs = a.T * a.top;
    constexpr uint16_t NONE = 0xFFFF;
#pragma unroll 1
    for (int i = threadIdx.x; i < a.E; i += threads) l.count[i] = 0;
    if (threadIdx.x == 0) l.start[0] = 0;
    // the thread's first pair's weight is on its way meanwhile
    const float w0 = threadIdx.x < pairs ? a.w[threadIdx.x] : 0.0f;
#pragma unroll 1
    for (int p = threadIdx.x; p < pairs; p += threads) {
        const uint32_t e = static_cast<uint32_t>(a.ids[p]);
        l.id[p] = e < static_cast<uint32_t>(a.E) ? static_cast<uint16_t>(e) : NONE;
    }
    __syncthreads();
#pragma unroll 1
    for (int p = threadIdx.x; p < pairs; p += threads) {
        const uint16_t e = l.id[p];
        bool first = e != NONE;
#pragma unroll 1
        for (int q = p - p % a.top; q < p; ++q) first &= l.id[q] != e;
        l.number[p] = first ? static_cast<uint8_t>(atomicAdd(&l.count[e], 1)) : 255;
    }
    __syncthreads();
    // a warp for 32 experts adds up those before them by itself
#pragma unroll 1
    for (int e0 = threadIdx.x & ~31; e0 < a.E; e0 += threads) {
        int base = 0, used = 0, most = 0;
#pragma unroll 1
        for (int e = lane; e < e0; e += 32) {
            const int c = l.count[e];
            base += c;
            used += c > 0;
            most = max(most, c);
        }
        const int e = e0 + lane, c = e < a.E ? l.count[e] : 0;
        most = max(most, c);
        base = __reduce_add_sync(0xFFFFFFFFu, base);
        used = __reduce_add_sync(0xFFFFFFFFu, used);
        int sum = base + c;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, k) - base;
            if (lane >= k) sum += v;
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, c > 0);
        if (e < a.E) l.start[e + 1] = sum;
        if (c > 0) l.busy[used + __popc(mask & ((1u << lane) - 1u))] = static_cast<uint16_t>(e);
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (e == a.E - 1) {
            l.experts[0] = used + __popc(mask);
            l.experts[1] = most;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int p = threadIdx.x; p < pairs; p += threads) {
        if (l.number[p] == 255) continue;
        const int e = l.id[p], t = p / a.top, at = l.start[e] + l.number[p];
        float w = p < threads ? w0 : a.w[p];
#pragma unroll 1
        for (int q = p + 1; q < (t + 1) * a.top; ++q)
            if (l.id[q] == e) w += a.w[q];
        l.pair[at] = static_cast<uint16_t>(p);
        l.token[at] = static_cast<uint16_t>(t);
        l.weight[at] = w;
    }
    __syncthreads();
}

}  // namespace bsfp8
