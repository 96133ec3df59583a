// moe_route.cuh -- the router of a mixture-of-experts layer: each token's `top` experts by
// their logits, their weights, and the rows in expert order.
//
//   ids[t][j]     expert of the j-th largest logit of token t; equal logits: the lower
//                 expert first; logits of -inf (and NaN) are closed and never taken
//   weights[t][j] softmax or sigmoid of the logits, over the chosen ones or over all
//   places[t][j]  where pair (t, j) stands among all pairs sorted by expert (stable)
//   rows[place]   the token there;  offsets[e] the first place of expert e
//
// What bounds it: one pass over the logits (16384 x 64 fp32: 4.2 MB), in practice latency and, for
// many experts, the selection's instructions: 1 token 3.7 us (a call 7.5, the host's time), 16384
// tokens, 4 of 64 11.2 us (two kernels), 16001 tokens, 8 of 256 18.8 (572 warp instructions a
// token, issue 61 % of the cycles).  A warp owns a token and a lane V
// neighbouring experts, so that the lowest lane of equal maxima holds the lowest expert.
//
// Up to two experts a lane: a pick is one warp maximum over the lanes' own maxima and one vote.
// More: the `top`-th largest of the lanes' own maxima is a bound that at least top logits reach
// and few others do; those that do (up to 32) come to a lane each, which counts the ones
// before it (16001 tokens, 8 of 256: 19 us; by picks of sorted lanes 22, of unsorted ones 37).
//
// Weights: expf, a sum over the lanes and __fdividef, off by 4.0e-8 to 6.7e-8 of the weights' norm
// (plain fp32 3.8e-8 to 6.0e-8); with correctly rounded quotients 3.8e-8 to 6.6e-8, and 16001
// tokens, 8 of 256 by sigmoids, take 19.5 us for 18.8.
//
// The expert order is a counting sort: integer counts of each CTA's tokens, and in the second
// kernel each CTA's base from the counts of the CTAs before it; nothing depends on the order in
// which atomics arrive.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "block128_rows.cuh"

namespace bsfp8 {

constexpr int ROUTE_THREADS = 1024, ROUTE_WARPS = ROUTE_THREADS / 32;
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
    int32_t *counts;          // [E][chunks]: pairs of each chunk's tokens
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

// What a lane has of a token's picks: the expert and key of pick `slot` (below top), or none.
struct Pick {
    int id, slot;
    uint32_t key, best;   // best: the largest key of all
};

// One pick after the other; pick j goes to lane j.  head: the lane's largest key.
template <int V>
__device__ __forceinline__ Pick pick_each(int top, uint32_t (&key)[V], uint32_t head) {
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    Pick r{-1, lane, 0u, 0u};
    int at = 0;
    for (int j = 0; j < top; ++j) {
        const uint32_t best = __reduce_max_sync(ALL, head);
        if (best == 0u) break;
        if (j == 0) r.best = best;
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
            r.id = e;
            r.key = best;
        }
    }
    return r;
}

// All picks at once, by a bound; false (and nothing done) where more than 32 keys reach it.
template <int V>
__device__ __forceinline__ bool pick_all(int top, const uint32_t (&key)[V], uint32_t head, uint2 *mine, Pick &r) {
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    uint32_t bound = 1u;   // fewer lanes than top with an open expert: every open one
    r = Pick{-1, 32, 0u, 0u};
    for (int j = 0; j < top; ++j) {
        const uint32_t best = __reduce_max_sync(ALL, head);
        if (j == 0) r.best = best;
        bound = max(best, 1u);
        if (best == 0u) break;
        if (lane == __ffs(__ballot_sync(ALL, head == best)) - 1) head = 0u;
    }
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += key[i] >= bound;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(ALL, sum, o);
        if (lane >= o) sum += v;
    }
    const int all = __shfl_sync(ALL, sum, 31);
    if (all > 32) return false;
    int at = sum - n;   // in the order of the experts
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (key[i] >= bound) mine[at++] = make_uint2(key[i], static_cast<uint32_t>(lane * V + i));
    __syncwarp();
    const uint2 own = lane < all ? mine[lane] : make_uint2(0u, 0u);
    __syncwarp();
    int before = 0;
    for (int c = 0; c < all; ++c) {
        const uint32_t k = __shfl_sync(ALL, own.x, c);
        before += k > own.x || (k == own.x && c < lane);
    }
    if (lane < all && before < top) {
        r.id = static_cast<int>(own.y);
        r.key = own.x;
        r.slot = before;
    }
    // slots without an expert go to lanes without one
    if (lane >= all && lane < top) r.slot = lane;
    return true;
}

// Picks and weights of a token; returns the lane's expert (-1: none).
template <int V>
__device__ __forceinline__ int route_token(const RouteArgs &a, int64_t token, uint32_t (&key)[V], uint2 *mine) {
    constexpr uint32_t ALL = 0xFFFFFFFFu;
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
    Pick r;
    if constexpr (V <= 2) {
        r = pick_each<V>(a.top, key, head);
    } else {
        if (!pick_all<V>(a.top, key, head, mine, r)) r = pick_each<V>(a.top, key, head);
    }
    const float v = key_logit(r.key), top = key_logit(r.best);
    float p = 0.0f;
    if (!a.sigmoid) {
        p = exp_below(v, top);
    } else {   // over the chosen ones: all scaled by exp(-m), m the largest below 0, so that their sum is not lost
        const float e = expf(-fabsf(v)), m = a.all ? 0.0f : fminf(top, 0.0f);
        p = __fdividef(m < 0.0f ? expf(v - m) : v > 0.0f ? 1.0f : e, 1.0f + e);
    }
    if (!r.key) p = 0.0f;
    if (!a.all) {
        sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
    }
    if (r.slot < a.top) {
        const bool divide = !a.all || !a.sigmoid;
        a.ids[token * a.top + r.slot] = r.id;
        a.weights[token * a.top + r.slot] = r.key ? (divide ? __fdividef(p, sum) : p) * a.scale : 0.0f;   // sum is in [0.5, E]
    }
    return r.id;
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
__device__ __forceinline__ void warp_pairs(int p0, int p1, int warp, int &lo, int &hi) {
    const int per = (p1 - p0 + ROUTE_WARPS - 1) / ROUTE_WARPS;
    lo = min(p1, p0 + warp * per);
    hi = min(p1, lo + per);
}

// Words of a row of wh: E and the total, an odd number, so that a column meets all banks.
__host__ __device__ constexpr int route_ld(int E) { return (E + 1) | 1; }

// wh[warp][e] += the warp's pairs of each expert.
__device__ __forceinline__ void count_pairs(const RouteArgs &a, int p0, int p1, int *wh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *mine = wh + warp * route_ld(a.E);
    int lo, hi;
    warp_pairs(p0, p1, warp, lo, hi);
    for (int p = lo + lane; p - lane < hi; p += 32) {
        const int e = p < hi ? a.ids[p] : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
}

// Places and rows of the CTA's pairs; base[e] + wh[warp][e] is the next place there.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, int p0, int p1, int *wh, const int *base) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *mine = wh + warp * route_ld(a.E);
    int lo, hi;
    warp_pairs(p0, p1, warp, lo, hi);
    for (int p = lo + lane; p - lane < hi; p += 32) {
        const int e = p < hi ? a.ids[p] : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const int at = e >= 0 ? base[e] + mine[e] + __popc(same & ((1u << lane) - 1u)) : -1;
        __syncwarp();
        if (e >= 0) {
            if (lane == __ffs(same) - 1) mine[e] += __popc(same);
            a.rows[at] = static_cast<int>(static_cast<uint32_t>(p) / static_cast<uint32_t>(a.top));
        }
        if (p < hi) a.places[p] = at;
        __syncwarp();
    }
}

// The rows from the number of pairs with an expert on, shared out over the CTAs.
__device__ __forceinline__ void fill_rows(const RouteArgs &a, int used) {
    for (int p = used + static_cast<int>(blockIdx.x * ROUTE_THREADS + threadIdx.x); p < a.T * a.top;
         p += static_cast<int>(gridDim.x * ROUTE_THREADS))
        a.rows[p] = -1;
}

// wh[w][e] of each warp w becomes `first` and what the warps before it have; returns all of them.
__device__ __forceinline__ int warp_starts(int *wh, int ld, int e, int first) {
    static_assert(ROUTE_WARPS == 32, "a lane for each warp");
    const int lane = threadIdx.x & 31, x = wh[lane * ld + e];
    int sum = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += y;
    }
    wh[lane * ld + e] = first + sum - x;
    return __shfl_sync(0xFFFFFFFFu, sum, 31);
}

constexpr int route_smem(int E) { return ((ROUTE_WARPS + 1) * route_ld(E) + (E + 1 + 31) / 32) * 4; }

// Picks of a CTA's tokens.  With an order: their counts, or, when there is one CTA, the
// whole order.
template <int V, bool BF16>
__global__ void __launch_bounds__(ROUTE_THREADS, 1) bsfp8_route_pick(const RouteArgs a) {
    extern __shared__ int sh[];   // wh[ROUTE_WARPS][ld], base[ld], seg
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = a.E + 1, ld = route_ld(a.E);
    int *wh = sh, *base = sh + ROUTE_WARPS * ld, *seg = base + ld;
    __shared__ uint2 candidates[V > 2 ? ROUTE_WARPS : 1][32];
    uint2 *mine = candidates[V > 2 ? warp : 0];
    const int t0 = static_cast<int>(blockIdx.x) * a.chunk, t1 = min(a.T, t0 + a.chunk);
    const bool one = a.offsets && gridDim.x == 1;
    if (a.offsets)
        for (int i = threadIdx.x; i < (one ? (ROUTE_WARPS + 1) * ld : ld); i += ROUTE_THREADS) (one ? wh : base)[i] = 0;
    wait_for_previous();
    launch_dependents();
    __syncthreads();
    for (int t = t0 + warp; t < t1; t += ROUTE_WARPS) {
        uint32_t key[V];
        load_keys<V, BF16>(a, t, key);
        const int id = route_token<V>(a, t, key, mine);
        if (a.offsets && !one && id >= 0) atomicAdd(&base[id], 1);
    }
    if (!a.offsets) return;
    __syncthreads();
    if (!one) {
        for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS)
            a.counts[e * a.chunks + blockIdx.x] = base[e];
        return;
    }
    const int pairs = a.T * a.top;   // below 2^30
    count_pairs(a, 0, pairs, wh);
    __syncthreads();
    for (int e = warp; e < a.E; e += ROUTE_WARPS) {
        const int total = warp_starts(wh, ld, e, 0);
        if (lane == 0) base[e] = total;
    }
    __syncthreads();
    scan_exclusive(base, n, seg);
    for (int e = threadIdx.x; e < n; e += ROUTE_THREADS) a.offsets[e] = base[e];
    fill_rows(a, base[a.E]);
    place_pairs(a, 0, pairs, wh, base);
}

// The order of the pairs of chunk blockIdx.x from the counts of all chunks.
__global__ void __launch_bounds__(ROUTE_THREADS, 1) bsfp8_route_order(const RouteArgs a) {
    extern __shared__ int sh[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = a.E + 1, ld = route_ld(a.E);
    int *wh = sh, *base = sh + ROUTE_WARPS * ld, *seg = base + ld;
    const int p0 = static_cast<int>(blockIdx.x) * a.chunk * a.top, p1 = min(a.T * a.top, p0 + a.chunk * a.top);
    for (int i = threadIdx.x; i < (ROUTE_WARPS + 1) * ld; i += ROUTE_THREADS) wh[i] = 0;
    wait_for_previous();
    launch_dependents();
    __syncthreads();
    count_pairs(a, p0, p1, wh);
    __syncthreads();
    // a warp for four experts at a time: all of each, what the chunks before this one have of it,
    // and (a lane for each warp's part) where the warps' pairs start
    constexpr int LOADS = (ROUTE_CHUNKS + 31) / 32;
    for (int e0 = warp * 4; e0 < a.E; e0 += ROUTE_WARPS * 4) {
        int x[4][LOADS];
        const int32_t *from = a.counts + e0 * a.chunks + lane;   // below 2^18
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                x[k][i] = e0 + k < a.E && lane + 32 * i < a.chunks ? from[k * a.chunks + 32 * i] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (e0 + k >= a.E) break;
            int all = 0, before = 0;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                all += x[k][i];
                before += lane + 32 * i < static_cast<int>(blockIdx.x) ? x[k][i] : 0;
            }
            all = __reduce_add_sync(0xFFFFFFFFu, all);
            before = __reduce_add_sync(0xFFFFFFFFu, before);
            warp_starts(wh, ld, e0 + k, before);
            if (lane == 0) base[e0 + k] = all;
        }
    }
    __syncthreads();
    scan_exclusive(base, n, seg);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < n; e += ROUTE_THREADS) a.offsets[e] = base[e];
    fill_rows(a, base[a.E]);
    place_pairs(a, p0, p1, wh, base);
}

}  // namespace bsfp8
