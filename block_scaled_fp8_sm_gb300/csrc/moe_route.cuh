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
// pick is one warp maximum over the lanes' own maxima and one vote.  A lane's own experts are
// sorted first, up to eight of them, so that its next maximum is a shift (16001 tokens, 8 of 256:
// searching them again for each pick took twice the instructions).  The expert order is a
// counting sort: integer counts of each CTA's tokens, and in the second kernel each CTA's
// base from the counts of the CTAs before it; nothing depends on the order in which atomics
// arrive.
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

// Sorts the lane's keys, the largest first, and their numbers (four bits each in `at`) with
// them; returns false where equal keys may be out of order.  Merge exchange (Batcher, 1968;
// Knuth, The Art of Computer Programming 3, 5.2.2, algorithm M).
template <int V>
__device__ __forceinline__ bool sort_keys(uint32_t (&key)[V], uint32_t &at) {
    uint32_t n[V];
#pragma unroll
    for (int i = 0; i < V; ++i) n[i] = i;
#pragma unroll
    for (int p = V / 2; p > 0; p /= 2) {
        int q = V / 2, r = 0, d = p;
#pragma unroll
        for (int step = 0; step < 4; ++step) {
            if (d > 0) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i + d < V && (i & p) == r) {
                        const bool swap = key[i + d] > key[i];
                        const uint32_t hi = max(key[i], key[i + d]), lo = min(key[i], key[i + d]);
                        const uint32_t a = swap ? n[i + d] : n[i], b = swap ? n[i] : n[i + d];
                        key[i] = hi, key[i + d] = lo, n[i] = a, n[i + d] = b;
                    }
                if (q == p) break;
                d = q - p;
                q /= 2;
                r = p;
            }
        }
    }
    at = 0u;
    bool distinct = true;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        at |= n[i] << (4 * i);
        if (i > 0) distinct &= key[i] != key[i - 1] || key[i] == 0u;
    }
    return distinct;
}

// A token's picks: lane j < top gets pick j, its expert (-1: none left) and its key.
template <int V>
__device__ __forceinline__ void pick(const RouteArgs &a, uint32_t (&key)[V], uint32_t head, int &id, uint32_t &mine) {
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    id = -1;
    mine = 0u;
    uint32_t at = 0u;
    bool sorted = false;
    if constexpr (V >= 2 && V <= 8) {
        uint32_t k[V];
#pragma unroll
        for (int i = 0; i < V; ++i) k[i] = key[i];
        sorted = __all_sync(ALL, sort_keys<V>(k, at));
        if (sorted) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = k[i];
        }
    }
    if (sorted) {
        for (int j = 0; j < a.top; ++j) {
            const uint32_t best = __reduce_max_sync(ALL, key[0]);
            if (best == 0u) break;
            const int src = __ffs(__ballot_sync(ALL, key[0] == best)) - 1;
            const int e = src * V + (__shfl_sync(ALL, at, src) & 15);
            if (lane == src) {
#pragma unroll
                for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
                key[V - 1] = 0u;
                at >>= 4;
            }
            if (lane == j) {
                id = e;
                mine = best;
            }
        }
        return;
    }
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
}

// Picks and weights of a token, written by lane j < top; returns its expert.
template <int V>
__device__ __forceinline__ int route_token(const RouteArgs &a, int64_t token, uint32_t (&key)[V]) {
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
    int id;
    uint32_t mine;
    pick<V>(a, key, head, id, mine);
    const float v = key_logit(mine), top = __shfl_sync(ALL, v, 0);
    float p = 0.0f;
    if (!a.sigmoid) {
        p = exp_below(v, top);
    } else {   // over the chosen ones: all scaled by exp(-m), m the largest below 0, so that their sum is not lost
        const float e = expf(-fabsf(v)), m = a.all ? 0.0f : fminf(top, 0.0f);
        p = (m < 0.0f ? expf(v - m) : v > 0.0f ? 1.0f : e) / (1.0f + e);
    }
    if (!mine) p = 0.0f;
    if (!a.all) {
        sum = p;
        for (int o = 1; o < a.top; o <<= 1) sum += __shfl_xor_sync(ALL, sum, o);   // the lanes from top on have zeros
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

// Places and rows of the CTA's pairs; wh[warp][e] is the next place there.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, int p0, int p1, int *wh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *mine = wh + warp * route_ld(a.E);
    int lo, hi;
    warp_pairs(p0, p1, warp, lo, hi);
    for (int p = lo + lane; p - lane < hi; p += 32) {
        const int e = p < hi ? a.ids[p] : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const int at = e >= 0 ? mine[e] + __popc(same & ((1u << lane) - 1u)) : -1;
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
        const int id = route_token<V>(a, t, key);
        if (a.offsets && !one && id >= 0) atomicAdd(&base[id], 1);
    }
    if (!a.offsets) return;
    __syncthreads();
    if (!one) {
        for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS)
            a.counts[static_cast<int64_t>(e) * a.chunks + blockIdx.x] = base[e];
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
    for (int i = threadIdx.x; i < ROUTE_WARPS * ld; i += ROUTE_THREADS) wh[i] += base[i % ld];
    for (int e = threadIdx.x; e < n; e += ROUTE_THREADS) a.offsets[e] = base[e];
    fill_rows(a, base[a.E]);
    __syncthreads();
    place_pairs(a, 0, pairs, wh);
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
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int c = lane + 32 * i;
                x[k][i] = e0 + k < a.E && c < a.chunks ? a.counts[static_cast<int64_t>(e0 + k) * a.chunks + c] : 0;
            }
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
    for (int i = threadIdx.x; i < ROUTE_WARPS * ld; i += ROUTE_THREADS) wh[i] += base[i % ld];
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < n; e += ROUTE_THREADS) a.offsets[e] = base[e];
    fill_rows(a, base[a.E]);
    __syncthreads();
    place_pairs(a, p0, p1, wh);
}

}  // namespace bsfp8
