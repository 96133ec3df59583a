// moe_route.cuh -- the router of a mixture-of-experts layer: each token's `top` experts by
// their logits, their weights, and the rows in expert order.
//
//   ids[t][j]     expert of the j-th largest logit of token t; equal logits: the lower
//                 expert first; logits of -inf (and NaN) are closed and never taken
//   weights[t][j] softmax or sigmoid of the logits, over the chosen ones or over all
//   places[t][j]  where pair (t, j) stands among all pairs sorted by expert (stable)
//   rows[place]   the token there;  offsets[e] the first place of expert e
//
// What bounds it: one pass over the logits (16384 x 64 fp32: 4.2 MB), in practice the
// selection's instructions and, for few tokens, latency.  A warp owns a token and a lane V
// neighbouring experts, so that the lowest lane of equal maxima holds the lowest expert: a
// pick is one warp maximum over the lanes' own maxima and one vote.  The expert order is a
// counting sort: integer counts of each CTA's tokens, and in the second kernel each CTA's
// base from the counts of the CTAs before it; nothing depends on the order in which atomics
// arrive.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "block128_rows.cuh"

namespace bsfp8 {

constexpr int ROUTE_THREADS = 512, ROUTE_WARPS = ROUTE_THREADS / 32;
constexpr int ROUTE_MAX_TOP = 32;       // a lane for each pick
constexpr int ROUTE_CHUNKS = 152;       // CTAs of the ordered form: one for each SM

struct RouteArgs {
    const void *logits;       // [T, E], rows of ld values
    int64_t ld;
    float *weights;           // [T, top]
    int32_t *ids;             // [T, top]
    int32_t *offsets;         // [E + 1], or null: no order
    int32_t *rows;            // [T * top]
    int32_t *places;          // [T, top]
    int32_t *counts;          // [E + 1][chunks]: pairs of each chunk's tokens (the last: without an expert)
    int T, E, top, chunk, chunks;   // chunk: tokens of a CTA
    int sigmoid, all, vec;    // all: weights over all experts; vec: rows allow vector loads
    float scale;
};

// Order-preserving key of a logit: 0 for -inf and NaN, larger for larger values; -0 = +0.
__device__ __forceinline__ uint32_t logit_key(float x) {
    x += 0.0f;
    const uint32_t u = __float_as_uint(x);
    const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
    return x > -INFINITY ? k : 0u;
}

__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The lane's V logits of a token: experts V lane ..
template <int V, bool BF16>
__device__ __forceinline__ void load_keys(const RouteArgs &a, int64_t token, uint32_t (&key)[V]) {
    const int e0 = static_cast<int>(threadIdx.x & 31) * V;
    if constexpr (BF16) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.logits) + token * a.ld + e0;
        if (V > 1 && a.vec) {
            constexpr int W = V < 8 ? V : 8;   // values of a load
#pragma unroll
            for (int i = 0; i < V; i += W) {
                uint32_t w[W / 2 + 1];
                const bool in = e0 + i < a.E;
                if constexpr (W == 8) {
                    const uint4 v = in ? *reinterpret_cast<const uint4 *>(p + i) : make_uint4(0u, 0u, 0u, 0u);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                } else if constexpr (W == 4) {
                    const uint2 v = in ? *reinterpret_cast<const uint2 *>(p + i) : make_uint2(0u, 0u);
                    w[0] = v.x, w[1] = v.y;
                } else {
                    w[0] = in ? *reinterpret_cast<const uint32_t *>(p + i) : 0u;
                }
#pragma unroll
                for (int j = 0; j < W; ++j)
                    key[i + j] = in ? logit_key(j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2])) : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = e0 + i < a.E ? logit_key(__bfloat162float(p[i])) : 0u;
        }
    } else {
        const float *p = static_cast<const float *>(a.logits) + token * a.ld + e0;
        if (V > 1 && a.vec) {
            constexpr int W = V < 4 ? V : 4;
#pragma unroll
            for (int i = 0; i < V; i += W) {
                float w[W + 1];
                const bool in = e0 + i < a.E;
                if constexpr (W == 4) {
                    const float4 v = in ? *reinterpret_cast<const float4 *>(p + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                } else {
                    const float2 v = in ? *reinterpret_cast<const float2 *>(p + i) : make_float2(0.f, 0.f);
                    w[0] = v.x, w[1] = v.y;
                }
#pragma unroll
                for (int j = 0; j < W; ++j) key[i + j] = in ? logit_key(w[j]) : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = e0 + i < a.E ? logit_key(p[i]) : 0u;
        }
    }
}

// exp(v - m) with m the row's largest; v == m covers a row of infinities.
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.0f : expf(v - m); }

// A token's picks: lane j < top writes pick j and returns its expert (-1: none left).
template <int V>
__device__ __forceinline__ int pick(const RouteArgs &a, int64_t token, uint32_t (&key)[V]) {
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    uint32_t head = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) head = max(head, key[i]);
    float sum = 0.0f;
    if (a.all && !a.sigmoid) {   // the softmax's sum over every open expert
        const float m = key_logit(__reduce_max_sync(ALL, head));
#pragma unroll
        for (int i = 0; i < V; ++i) sum += key[i] ? exp_below(key_logit(key[i]), m) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
    }
    int id = -1, at = 0;
    uint32_t mine = 0u;
    for (int j = 0; j < a.top; ++j) {
        const uint32_t best = __reduce_max_sync(ALL, head);
        if (best == 0u) break;
        const int src = __ffs(__ballot_sync(ALL, head == best)) - 1;
        if (lane == src) {   // the lowest of its experts with this value is taken
            bool taken = false;
            head = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool hit = !taken && key[i] == best;
                taken |= hit;
                if (hit) at = i;
                key[i] = hit ? 0u : key[i];
                head = max(head, key[i]);
            }
        }
        const int e = src * V + __shfl_sync(ALL, at, src);
        if (lane == j) {
            id = e;
            mine = best;
        }
    }
    const float v = key_logit(mine), top = __shfl_sync(ALL, v, 0);
    float p = 0.0f;
    if (mine) {
        if (!a.sigmoid) {
            p = exp_below(v, top);
        } else if (v > 0.0f) {
            p = 1.0f / (1.0f + expf(-v));
        } else {   // over the chosen ones: all scaled by exp(-m), so that their sum is not lost
            const float m = a.all ? 0.0f : fminf(top, 0.0f);
            p = expf(v - m) / (1.0f + expf(v));
        }
    }
    if (!a.all) {
        sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
    }
    if (lane < a.top) {
        const bool divide = !a.all || !a.sigmoid;
        a.ids[token * a.top + lane] = id;
        a.weights[token * a.top + lane] = mine ? (divide ? p / sum : p) * a.scale : 0.0f;
    }
    return id;
}

// Exclusive sums of v[0 .. n) in place, by the whole CTA; seg: a word for each 32 of them.
__device__ __forceinline__ void scan_exclusive(int *v, int n, int *seg) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, segs = (n + 31) / 32;
    for (int s = warp; s < segs; s += ROUTE_WARPS) {
        const int i = s * 32 + lane, x = i < n ? v[i] : 0;
        int sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        if (i < n) v[i] = sum - x;
        if (lane == 31) seg[s] = sum;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += ROUTE_THREADS) {
        int base = 0;
        for (int s = 0; s < i / 32; ++s) base += seg[s];
        v[i] += base;
    }
    __syncthreads();
}

// The pairs of warp `warp` of a CTA's [p0, p1): contiguous, so that the order is stable.
__device__ __forceinline__ void warp_pairs(int64_t p0, int64_t p1, int warp, int64_t &lo, int64_t &hi) {
    const int64_t per = (p1 - p0 + ROUTE_WARPS - 1) / ROUTE_WARPS;
    lo = min(p1, p0 + warp * per);
    hi = min(p1, lo + per);
}

// wh[warp][bucket] += the warp's pairs of each bucket (E: without an expert).
__device__ __forceinline__ void count_pairs(const RouteArgs &a, int64_t p0, int64_t p1, int *wh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *mine = wh + warp * (a.E + 1);
    int64_t lo, hi;
    warp_pairs(p0, p1, warp, lo, hi);
    for (int64_t p = lo + lane; p - lane < hi; p += 32) {
        int e = p < hi ? a.ids[p] : -2;
        if (e == -1) e = a.E;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
}

// Places and rows of the CTA's pairs; wh[warp][bucket] is the next place there.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, int64_t p0, int64_t p1, int *wh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *mine = wh + warp * (a.E + 1);
    int64_t lo, hi;
    warp_pairs(p0, p1, warp, lo, hi);
    for (int64_t p = lo + lane; p - lane < hi; p += 32) {
        int e = p < hi ? a.ids[p] : -2;
        const bool none = e == -1;
        if (none) e = a.E;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const int at = e >= 0 ? mine[e] + __popc(same & ((1u << lane) - 1u)) : 0;
        __syncwarp();
        if (e >= 0) {
            if (lane == __ffs(same) - 1) mine[e] += __popc(same);
            a.rows[at] = none ? -1 : static_cast<int32_t>(p / a.top);
            a.places[p] = none ? -1 : at;
        }
        __syncwarp();
    }
}

constexpr int route_smem(int E) { return ((ROUTE_WARPS + 1) * (E + 1) + (E + 1 + 31) / 32) * 4; }

// Picks of a CTA's tokens.  With an order: their counts, or, when there is one CTA, the
// whole order.
template <int V, bool BF16>
__global__ void __launch_bounds__(ROUTE_THREADS) bsfp8_route_pick(const RouteArgs a) {
    extern __shared__ int sh[];   // wh[ROUTE_WARPS][E + 1], base[E + 1], seg
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = a.E + 1;
    int *wh = sh, *base = sh + ROUTE_WARPS * n, *seg = base + n;
    const int t0 = static_cast<int>(blockIdx.x) * a.chunk, t1 = min(a.T, t0 + a.chunk);
    const bool one = a.offsets && gridDim.x == 1;
    if (a.offsets)
        for (int i = threadIdx.x; i < (one ? (ROUTE_WARPS + 1) * n : n); i += ROUTE_THREADS)
            (one ? wh : base)[i] = 0;
    wait_for_previous();
    launch_dependents();
    __syncthreads();
    for (int t = t0 + warp; t < t1; t += ROUTE_WARPS) {
        uint32_t key[V];
        load_keys<V, BF16>(a, t, key);
        const int id = pick<V>(a, t, key);
        if (a.offsets && !one && lane < a.top) atomicAdd(&base[id < 0 ? a.E : id], 1);
    }
    if (!a.offsets) return;
    __syncthreads();
    if (!one) {
        for (int e = threadIdx.x; e < n; e += ROUTE_THREADS)
            a.counts[static_cast<int64_t>(e) * a.chunks + blockIdx.x] = base[e];
        return;
    }
    const int64_t pairs = static_cast<int64_t>(a.T) * a.top;
    count_pairs(a, 0, pairs, wh);
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += ROUTE_THREADS) {
        int sum = 0;
        for (int w = 0; w < ROUTE_WARPS; ++w) sum += wh[w * n + e];
        base[e] = sum;
    }
    __syncthreads();
    scan_exclusive(base, n, seg);
    for (int e = threadIdx.x; e < n; e += ROUTE_THREADS) {
        int at = base[e];
        a.offsets[e] = at;
        for (int w = 0; w < ROUTE_WARPS; ++w) {
            const int c = wh[w * n + e];
            wh[w * n + e] = at;
            at += c;
        }
    }
    __syncthreads();
    place_pairs(a, 0, pairs, wh);
}

// The order of the pairs of chunk blockIdx.x from the counts of all chunks.
__global__ void __launch_bounds__(ROUTE_THREADS) bsfp8_route_order(const RouteArgs a) {
    extern __shared__ int sh[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = a.E + 1;
    int *wh = sh, *base = sh + ROUTE_WARPS * n, *seg = base + n;
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.chunk * a.top;
    const int64_t p1 = min(static_cast<int64_t>(a.T) * a.top, p0 + static_cast<int64_t>(a.chunk) * a.top);
    for (int i = threadIdx.x; i < ROUTE_WARPS * n; i += ROUTE_THREADS) wh[i] = 0;
    wait_for_previous();
    launch_dependents();
    __syncthreads();
    count_pairs(a, p0, p1, wh);
    __syncthreads();
    // a warp for each bucket: all of it, and what the chunks before this one have of it
    for (int e = warp; e < n; e += ROUTE_WARPS) {
        int all = 0, before = 0;
        for (int c = lane; c < a.chunks; c += 32) {
            const int x = a.counts[static_cast<int64_t>(e) * a.chunks + c];
            all += x;
            if (c < static_cast<int>(blockIdx.x)) before += x;
        }
        all = __reduce_add_sync(0xFFFFFFFFu, all);
        before = __reduce_add_sync(0xFFFFFFFFu, before);
        if (lane == 0) {
            base[e] = all;
            int at = before;   // relative to the bucket's first place, which is known after the scan
            for (int w = 0; w < ROUTE_WARPS; ++w) {
                const int x = wh[w * n + e];
                wh[w * n + e] = at;
                at += x;
            }
        }
    }
    __syncthreads();
    scan_exclusive(base, n, seg);
    for (int i = threadIdx.x; i < ROUTE_WARPS * n; i += ROUTE_THREADS) wh[i] += base[i % n];
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < n; e += ROUTE_THREADS) a.offsets[e] = base[e];
    __syncthreads();
    place_pairs(a, p0, p1, wh);
}

}  // namespace bsfp8
