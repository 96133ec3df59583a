// moe_tile.cuh -- the mixture-of-experts layer of moe_layer.cuh for more than eight tokens,
// on the tensor cores (tcgen05): the weights come by TMA and are never touched by a register.
//
// A weight tile's 128 rows are the MMA's M side, an expert's tokens its N side, in E4M3: a
// number v of the activations becomes two (x) or three (h) codes,
//   v / s = q0 + q1 / 32 + q2 / 1024,   each the nearest E4M3 of what the ones before leave,
// s the power of two that brings the largest of the token's 128 values of a K block to
// [2^7, 2^8).  Each code takes four of v's bits, so two hold the 8 bits of a bf16 exactly
// (down to 2^-14 of the block's largest; below, the error stays under 2^-22 of it), and
// three hold 12 bits of h.  The block-scaled MMA adds the codes' products with their powers
// of 32 (constant UE8M0 scales in tensor memory), and the epilogue adds (s_w s) times the sum
// of a 128-K block to fp32 registers.  The tensor cores are far from busy: the call is bound
// by the weights' bytes.
//
// Roles (384 threads): warp 0 TMA, warp 1 MMA (one lane each), warps 4-7 epilogue (a thread
// owns a row of the tile and all tokens), up to six of the others make the codes, each a stage
// in turn, so that the latency of its loads is spread over six stages.
//
// Up: a tile is 64 columns of h, 16 gate rows and 16 up rows in turn, so that a warp holds
// both; CTAs take tiles in turn.  Down: a tile is 128 columns of the output with all busy
// experts one after the other, summed in shared memory; the stages of all tiles are one
// line, cut into equal pieces for the CTAs.  Where a cut goes through a tile, the parts go to
// the workspace and the CTA that comes last adds them in order: no CTA waits for another,
// and calls repeat bit for bit.
//
// Every wait is bounded as in the other kernels.
#pragma once
#include "block128_tile.cuh"
#include "moe_layer.cuh"
#include "quant_math.cuh"

namespace bsfp8 {

constexpr int MT_THREADS = 384;
constexpr int MT_CTAS = 152;           // one for each SM
constexpr int MT_MAX_STAGES = 6;
constexpr int MT_MAKERS = 6;           // warps that make codes
constexpr int MT_SX_RING = 32;         // slots of scales: the K blocks of all stages and partials, and more
constexpr int MT_SMEM = 232448;        // all that a CTA can have

struct MoeTileArgs : MoeArgs {
    CUtensorMap tmW;
    float *part;              // [2 MT_CTAS][T][128]: sums of the tiles that a cut goes through
    int *counters;            // [MT_CTAS]: parts of the tile that starts in this CTA and goes on
    uint32_t *status;
    long long wait_limit;
    int ring;                 // bytes of shared memory for the stages
};

// DOWN, NG: groups of eight tokens that an expert can have.
template <bool DOWN, int NG>
struct CfgMoe {
    static constexpr int PIECES = DOWN ? 3 : 2;
    static constexpr int A_BYTES = 128 * 128;   // weights of a K block; a stage has two
    // Tensor memory: partials of 8 NG columns for each of a stage's blocks, then 4 columns of
    // scales for each code
    static constexpr int STRIDE = 16 * NG;
    static constexpr int BUFS = NG == 8 ? 3 : 4;
    static constexpr int SF = BUFS * STRIDE;
    static constexpr int COLS = NG == 2 ? 256 : 512;
};

template <bool DOWN, int NG>
struct CtrlMoe {
    uint64_t full[MT_MAX_STAGES], empty[MT_MAX_STAGES];   // full: the weights and the codes
    uint64_t tfull[4], tempty[4], drain;
    uint32_t tmem;
    int abort, last;
    alignas(16) uint32_t sf[3][32];                     // the codes' scales: 1, 2^-5, 2^-10 as UE8M0 bytes
    alignas(16) float sx[MT_SX_RING][8 * NG];   // read four at a time
    alignas(16) float sums[DOWN ? 8 * NG : 1][128];
};

// Shared memory beside the stages, which get the rest.
template <bool DOWN, int NG>
inline int smem_moe_fixed(int T, int top, int E) {
    return 1024 + moe_pad16(static_cast<int>(sizeof(CtrlMoe<DOWN, NG>))) + moe_lists_layout(T, top, E).bytes;
}

template <typename Ctl>
__device__ __forceinline__ bool wait_moe(uint64_t *bar, uint32_t parity, Ctl *ctl, const MoeTileArgs &a) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0u) {
            if (*reinterpret_cast<volatile int *>(&ctl->abort)) return false;
            if (clock64() - t0 > a.wait_limit) {
                *reinterpret_cast<volatile int *>(&ctl->abort) = 1;
                atomicOr(a.status, STATUS_TIMEOUT);
                return false;
            }
        }
    }
}

// A run of stages (two 128-K blocks each) of one expert in one tile.
struct MoeSeg {
    int b, c, k0, k1;   // number of the busy expert, tile, stages [k0, k1) of its K
    bool end;           // the tile's last
};

// The segments of this CTA in order; every role walks them alike.
template <bool DOWN>
struct MoeWalk {
    int64_t pos, end, all;   // down: the stages of all tiles,
    int ctas;                // and the CTAs that have some
    int busy, KS, tiles;     // KS: stages of a tile's K

    __device__ __forceinline__ MoeWalk(int busy_, int KS_, int tiles_) : busy(busy_), KS(KS_), tiles(tiles_) {
        if constexpr (DOWN) {
            all = static_cast<int64_t>(tiles) * busy * KS;
            ctas = static_cast<int>(min(all, static_cast<int64_t>(gridDim.x)));
            const bool in = static_cast<int>(blockIdx.x) < ctas;
            pos = in ? all * blockIdx.x / ctas : 0;
            end = in ? all * (blockIdx.x + 1) / ctas : 0;
        } else {
            pos = blockIdx.x;
            end = static_cast<int64_t>(tiles) * busy;
        }
    }
    __device__ __forceinline__ bool next(MoeSeg &s) {
        if (pos >= end) return false;
        if constexpr (DOWN) {
            const int64_t per = static_cast<int64_t>(busy) * KS;
            const int64_t c = pos / per;
            const int in = static_cast<int>(pos - c * per);
            s.c = static_cast<int>(c);
            s.b = in / KS;
            s.k0 = in - s.b * KS;
            s.k1 = static_cast<int>(min(static_cast<int64_t>(KS), s.k0 + (end - pos)));
            s.end = s.b + 1 == busy && s.k1 == KS;
            pos += s.k1 - s.k0;
        } else {
            const int i = static_cast<int>(pos);
            s.b = i / tiles;
            s.c = i - s.b * tiles;
            s.k0 = 0;
            s.k1 = KS;
            s.end = true;
            pos += gridDim.x;
        }
        return true;
    }
};

// The power of two that brings amax to [2^7, 2^8), and its inverse (infinite for an infinite
// amax: the token's results are then not finite either).
__device__ __forceinline__ float scale_to_e4m3(float amax, float &inverse) {
    const uint32_t e = max(__float_as_uint(amax) >> 23, 8u);
    inverse = e == 255u ? amax : __uint_as_float((e - 7u) << 23);
    return __uint_as_float((261u - e) << 23);
}

// The next codes of four values, in v as fp16; v becomes what they leave, times 32.
__device__ __forceinline__ uint32_t take_codes(__half2 (&v)[2]) {
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "r"(*reinterpret_cast<const uint32_t *>(&v[0])), "r"(*reinterpret_cast<const uint32_t *>(&v[1])));
    const uint32_t a = half2_of_e4m3x2(w), b = half2_of_e4m3x2_hi(w);
    const __half2 k = __float2half2_rn(32.0f);
    v[0] = __hmul2(__hsub2(v[0], *reinterpret_cast<const __half2 *>(&a)), k);
    v[1] = __hmul2(__hsub2(v[1], *reinterpret_cast<const __half2 *>(&b)), k);
    return w;
}

// Scales of the weights' K blocks 2 k .. 2 k + 15 of a tile, one in a lane of each half of a
// warp; sw: those of the thread's row, which are the same for a half.
__device__ __forceinline__ float row_scales(const float *sw, int KB, int k) {
    return sw[min(2 * k + static_cast<int>(threadIdx.x & 15), KB - 1)];
}

__device__ __forceinline__ void store_bf16x4(__nv_bfloat16 *to, float4 v) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
}

// The epilogue's sum over the stages of a segment: acc[token].  next: its first scales.
template <bool DOWN, int NG, typename Ctl>
__device__ __forceinline__ bool sum_blocks(const MoeTileArgs &a, Ctl *ctl, float (&acc)[8 * NG], const MoeSeg &s,
                                           const float *sw, float next, int KB, int ng, uint32_t taddr, int &it, int &b,
                                           uint32_t &bph) {
    using C = CfgMoe<DOWN, NG>;
#pragma unroll
    for (int j = 0; j < 8 * NG; ++j) acc[j] = 0.0f;
    const int lane = threadIdx.x & 31;
    float have = 0.0f;
    for (int ks = s.k0; ks < s.k1; ++ks) {
        const int in = 2 * (ks - s.k0) & 15;
        if (in == 0) {
            have = next;
            next = row_scales(sw, KB, ks + 8);
        }
        const float w0 = __shfl_sync(0xFFFFFFFFu, have, (lane & 16) + in);
        const float w1 = __shfl_sync(0xFFFFFFFFu, have, (lane & 16) + in + 1);
        if (!__all_sync(0xFFFFFFFFu, wait_moe(&ctl->tfull[b], bph, ctl, a))) return false;
        tc_fence_after();
        const bool two = 2 * ks + 1 < KB;
        const float4 *sx0 = reinterpret_cast<const float4 *>(ctl->sx[2 * it % MT_SX_RING]);
        const float4 *sx1 = reinterpret_cast<const float4 *>(ctl->sx[(2 * it + 1) % MT_SX_RING]);
#pragma unroll
        for (int g = 0; g < NG; g += 2) {   // sixteen tokens at a time
            if (g < ng) {
                uint32_t p[16], r[16];
                tmem_ld_x16(taddr + b * C::STRIDE + 8 * g, p);
                if (two) tmem_ld_x16(taddr + b * C::STRIDE + 8 * NG + 8 * g, r);
                tmem_ld_wait_for(p);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 v = sx0[2 * g + j];
                    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[8 * g + 4 * j + k] = fmaf(w0 * f[k], __uint_as_float(p[4 * j + k]), acc[8 * g + 4 * j + k]);
                }
                if (two) {
                    tmem_ld_wait_for(r);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 v = sx1[2 * g + j];
                        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[8 * g + 4 * j + k] = fmaf(w1 * f[k], __uint_as_float(r[4 * j + k]), acc[8 * g + 4 * j + k]);
                    }
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tempty[b]);
        ++it;
        if (++b == C::BUFS) {
            b = 0;
            bph ^= 1u;
        }
    }
    return true;
}

template <bool DOWN, int NG>
__global__ void __launch_bounds__(MT_THREADS, 1) bsfp8_moe_tile(const __grid_constant__ MoeTileArgs a) {
    using C = CfgMoe<DOWN, NG>;
    using Ctl = CtrlMoe<DOWN, NG>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + a.ring);
    const MoeLists L = moe_lists(smem + a.ring + moe_pad16(static_cast<int>(sizeof(Ctl))), a.T, a.top, a.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < MT_MAX_STAGES; ++s) {
            mbar_init(&ctl->full[s], 3);   // the weights and the codes of two blocks
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(&ctl->tfull[b], 2);
            mbar_init(&ctl->tempty[b], 4);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.tmW);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem, C::COLS);
        tmem_relinquish();
    }
    if (warp == 2) {
#pragma unroll
        for (int i = 0; i < 3; ++i) ctl->sf[i][lane] = 0x7F7F7F7Fu - i * 0x05050505u;
        fence_proxy_async_smem();
    }
    // Down does not wait here: what it reads before its makers and epilogue wait (routing,
    // weights) is not written by the up kernel, and the kernels before that one had ended
    // when it let this one start.
    if constexpr (!DOWN) wait_for_previous();
    build_lists(a, L);
    if constexpr (!DOWN) {
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < MT_CTAS; i += MT_THREADS) a.counters[i] = 0;
        launch_dependents();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    // a stage: two K blocks of the weights' 128 rows, and the codes of as many tokens as an
    // expert has at most (rows of eight tokens for each code; the MMA takes an even number)
    const int busy = L.experts[0], most = (L.experts[1] + 7) / 8;
    const int code_bytes = (C::PIECES * most + (most & 1)) * 1024;   // of a block
    const int stage_bytes = 2 * (C::A_BYTES + code_bytes);
    const int stages = min(MT_MAX_STAGES, a.ring / stage_bytes);
    // Warps that make codes, a block each in turn.  Not more than all stages have blocks: a
    // maker that looked further ahead would meet an `empty` barrier two rounds behind, whose
    // parity says that the stage is free.
    const int makers = min(MT_MAKERS, 2 * stages);
    const int K = DOWN ? a.I : a.H, KB = (K + 127) / 128, KS = (KB + 1) / 2;
    const int tiles = DOWN ? (a.H + 127) / 128 : (a.I + 63) / 64;
    MoeWalk<DOWN> walk(busy, KS, tiles);
    const MoeWalk<DOWN> whole = walk;
    MoeSeg s;

    if (warp == 0) {
        if (elect_one()) {
            int it = 0, st = 0;
            uint32_t ph = 1;
            bool ok = true;
            while (ok && walk.next(s)) {
                const int e = L.busy[s.b];
                // up: pieces of 16 columns that exist
                const int pieces = DOWN ? 0 : min(4, (a.I - s.c * 64) / 16);
                for (int ks = s.k0; ks < s.k1; ++ks) {
                    ok = wait_moe(&ctl->empty[st], ph, ctl, a);
                    if (!ok) break;
                    const int blocks = min(2, KB - 2 * ks);
                    mbar_arrive_expect_tx(&ctl->full[st], blocks * (DOWN ? C::A_BYTES : pieces * 4096));
                    for (int h = 0; h < blocks; ++h) {
                        uint8_t *da = smem + st * stage_bytes + h * C::A_BYTES;
                        const int k = (2 * ks + h) * 128;
                        if constexpr (DOWN) {
                            tma_load_2d(&a.tmW, &ctl->full[st], da, k, e * a.H + s.c * 128);
                        } else {
                            for (int q = 0; q < pieces; ++q) {
                                const int row = e * 2 * a.I + s.c * 64 + q * 16;
                                tma_load_2d(&a.tmW, &ctl->full[st], da + q * 4096, k, row);
                                tma_load_2d(&a.tmW, &ctl->full[st], da + q * 4096 + 2048, k, row + a.I);
                            }
                        }
                    }
                    ++it;
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // no load is in flight when the CTA leaves (where codes are missing, after a wait
            // that ran out, the limit is the time that the loads get)
            const long long t0 = clock64();
            for (int d = max(0, it - stages); d < it; ++d) {
                while (!mbar_try_wait(&ctl->full[d % stages], static_cast<uint32_t>(d / stages) & 1u))
                    if (clock64() - t0 > a.wait_limit) break;
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < C::PIECES; ++i)
                tmem_cp_32x128b_warpx4(tmem + C::SF + 4 * i, sdesc_sf_lines(smem_u32(ctl->sf[i])));
            int st = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            bool ok = true, ready = false;
            while (ok && walk.next(s)) {
                const int e = L.busy[s.b], ng = (L.start[e + 1] - L.start[e] + 7) / 8;
                const uint32_t idesc = idesc_mxf8f6f4(128, (8 * ng + 15) / 16 * 16, 0, 0);
                for (int ks = s.k0; ks < s.k1; ++ks) {
                    const uint32_t at = smem_u32(smem + st * stage_bytes);
                    const uint64_t ad = sdesc_k_sw128(at), bd = sdesc_k_sw128(at + 2 * C::A_BYTES);
                    const int blocks = min(2, KB - 2 * ks);
                    ok = (ready || wait_moe(&ctl->full[st], ph, ctl, a)) && wait_moe(&ctl->tempty[b], bph, ctl, a);
                    if (!ok) break;
                    tc_fence_after();
                    uint64_t *empty = &ctl->empty[st];
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                    for (int h = 0; h < blocks; ++h) {
                        const uint64_t ah = ad + h * (C::A_BYTES / 16), bh = bd + h * (code_bytes / 16);
                        const uint32_t d = tmem + b * C::STRIDE + h * 8 * NG;
#pragma unroll
                        for (int p = 0; p < C::PIECES; ++p)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_mxf8(d, ah + 2 * i, bh + p * ng * 64 + 2 * i, idesc, tmem + C::SF, tmem + C::SF + 4 * p,
                                         (p | i) != 0);
                        // the next stage is looked for while the pipe is busy
                        if (h == 0) ready = mbar_test_wait(&ctl->full[st], ph);
                    }
                    mma_commit(&ctl->tfull[b]);
                    mma_commit(empty);
                    mbar_arrive(&ctl->tfull[b]);   // the makers' scales are before this
                    if (++b == C::BUFS) {
                        b = 0;
                        bph ^= 1u;
                    }
                }
            }
            // all MMAs have completed before tensor memory is freed
            mma_commit(&ctl->drain);
            const long long t0 = clock64();
            while (!mbar_try_wait(&ctl->drain, 0))
                if (clock64() - t0 > a.wait_limit) break;
        }
    } else if (warp < 4 || warp >= 8) {
        if constexpr (DOWN) wait_for_previous();
        // block `it` (two in a stage) is this warp's where it mod makers is its number; lane l makes the codes of the
        // values 4 l .. 4 l + 3 of each token, eight tokens at a time, the next ones in flight
        const int maker = warp < 4 ? warp - 2 : warp - 6;
        if (maker < makers) {
            int it = maker, st = maker / 2, kb = 0, k1 = 0, first = 0, n = 0;   // K blocks [kb, k1) of the segment are ahead
            uint32_t ph = 1;
            uint2 v[8];
            float hs[8];
            // `skip` blocks on, into the segments that follow
            auto advance = [&](int skip) {
                kb += skip;
                while (kb >= k1) {
                    const int over = kb - k1;
                    if (!walk.next(s)) return false;
                    kb = 2 * s.k0 + over;
                    k1 = 2 * s.k1;
                }
                const int e = L.busy[s.b];
                first = L.start[e];
                n = L.start[e + 1] - first;
                return true;
            };
            auto load = [&](int g) {
                const int k = kb * 128 + 4 * lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int m = 8 * g + i;
                    v[i] = make_uint2(0u, 0u);
                    hs[i] = 0.0f;
                    if (m < n && k < K) {   // K is a multiple of 16
                        if constexpr (DOWN) {
                            const int64_t pair = L.pair[first + m];
                            v[i] = *reinterpret_cast<const uint2 *>(a.h + pair * a.I + k);
                            hs[i] = a.hs[pair * (a.I / 16) + k / 16];
                        } else {
                            v[i] = *reinterpret_cast<const uint2 *>(a.x + static_cast<int64_t>(L.token[first + m]) * a.H + k);
                        }
                    }
                }
            };
            bool more = advance(maker);
            if (more) load(0);
            while (more) {
                if (!__all_sync(0xFFFFFFFFu, wait_moe(&ctl->empty[st], ph, ctl, a))) break;
                uint8_t *db = smem + st * stage_bytes + 2 * C::A_BYTES + (it & 1) * code_bytes;
                float *sx = ctl->sx[it % MT_SX_RING];
                const int rows = n, ng = (n + 7) / 8;
                for (int g = 0; g < ng; ++g) {
                    // fp16 with the block's largest in [2^7, 2^8): exact down to 2^-22 of it
                    __half2 f[8][2];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float inverse;
                        if constexpr (DOWN) {   // h's own scales (of the largest of 16 in [2^14, 2^15)) say enough
                            const float top = fmaxf(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(hs[i]))), 0x1p-126f);
                            const __half2 r = __float2half2_rn(hs[i] * __uint_as_float((247u << 23) - __float_as_uint(top)));
                            f[i][0] = __hmul2(*reinterpret_cast<const __half2 *>(&v[i].x), r);
                            f[i][1] = __hmul2(*reinterpret_cast<const __half2 *>(&v[i].y), r);
                            inverse = top < 0x1p114f ? top * 128.0f : INFINITY;   // 2^114: of an infinite h
                        } else {
                            uint32_t a0, a1;
                            asm("abs.bf16x2 %0, %1;" : "=r"(a0) : "r"(v[i].x));
                            asm("abs.bf16x2 %0, %1;" : "=r"(a1) : "r"(v[i].y));
                            asm("max.bf16x2 %0, %0, %1;" : "+r"(a0) : "r"(a1));
                            const uint32_t top = max(a0 << 16, a0 & 0xFFFF0000u);
                            const float sc = scale_to_e4m3(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top)), inverse);
                            f[i][0] = __floats2half2_rn(bf16_lo(v[i].x) * sc, bf16_hi(v[i].x) * sc);
                            f[i][1] = __floats2half2_rn(bf16_lo(v[i].y) * sc, bf16_hi(v[i].y) * sc);
                        }
                        if (lane == i) sx[8 * g + i] = inverse;
                    }
                    if (g + 1 < ng) {
                        load(g + 1);
                    } else {
                        more = advance(makers);
                        if (more) load(0);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (8 * g + i < rows) {
                            // row p * 8 ng + m of the stage; 16-byte pieces exchanged by the row's low bits
                            const int at = ((((lane >> 2) ^ i) << 4) | ((lane & 3) << 2)) + (8 * g + i) * 128;
#pragma unroll
                            for (int p = 0; p < C::PIECES; ++p)
                                *reinterpret_cast<uint32_t *>(db + p * ng * 1024 + at) = take_codes(f[i]);
                        }
                    }
                }
                fence_proxy_async_smem();   // the codes become visible to the MMA
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->full[st]);
                st += ((it & 1) + makers) >> 1;
                it += makers;
                if (st >= stages) {
                    st -= stages;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp >= 4) {
        if constexpr (DOWN) wait_for_previous();
        const int q = warp & 3, row = q * 32 + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
        int it = 0, b = 0;
        uint32_t bph = 0;
        bool ok = true;
        if constexpr (!DOWN) {
            const int NB = (2 * a.I + 127) / 128;
            const float *sw = a.s1;
            float scales = 0.0f;
            auto begin = [&](const MoeSeg &v) {   // a segment's first scales
                const int col = min(v.c * 64 + q * 16 + (lane & 15), a.I - 1);
                sw = a.s1 + (static_cast<int64_t>(L.busy[v.b]) * NB + ((lane < 16 ? 0 : a.I) + col) / 128) * KB;
                scales = row_scales(sw, KB, v.k0);
            };
            bool more = walk.next(s);
            if (more) begin(s);
            while (ok && more) {
                const int e = L.busy[s.b], first = L.start[e], n = L.start[e + 1] - first, ng = (n + 7) / 8;
                const int col = s.c * 64 + q * 16 + (lane & 15);   // lanes 0-15 hold its gate, 16-31 its up
                float acc[8 * NG];
                ok = sum_blocks<DOWN, NG>(a, ctl, acc, s, sw, scales, KB, ng, taddr, it, b, bph);
                if (!ok) break;
                more = walk.next(s);
                if (more) begin(s);   // on their way while this tile is finished
                const bool low = lane < 16;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    if (g < ng) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {   // lanes 0-15 take tokens 0-3 of the group, the others 4-7
                            const float mine = low ? acc[8 * g + j] : acc[8 * g + 4 + j];
                            const float give = low ? acc[8 * g + 4 + j] : acc[8 * g + j];
                            const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 16);
                            const float v = silu_mul(low ? mine : got, low ? got : mine);
                            float amax = fabsf(v);
#pragma unroll
                            for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                            float inverse;
                            const float sc = scale_to_half(amax, inverse);
                            const int m = 8 * g + j + (low ? 0 : 4);
                            if (m < n && col < a.I) {
                                const int64_t pair = L.pair[first + m];
                                a.h[pair * a.I + col] = __float2half_rn(v * sc);
                                if ((lane & 15) == 0) a.hs[pair * (a.I / 16) + col / 16] = inverse;
                            }
                        }
                    }
                }
            }
        } else {
            const int64_t per = static_cast<int64_t>(busy) * KS, all = walk.all, G = walk.ctas;
            const int NB = (a.H + 127) / 128;
            if (busy == 0)   // no token has an expert
                for (int c = blockIdx.x; c < tiles; c += gridDim.x)
                    for (int t = 0; t < a.T; ++t)
                        if (c * 128 + row < a.H) a.out[static_cast<int64_t>(t) * a.H + c * 128 + row] = __float2bfloat16_rn(0.0f);
            for (int t = 0; t < a.T; ++t) ctl->sums[t][row] = 0.0f;
            MoeSeg ahead;   // the next segment, whose first scales are on their way
            const float *sw = a.s2;
            float scales = 0.0f;
            auto begin = [&](const MoeSeg &v) {
                sw = a.s2 + (static_cast<int64_t>(L.busy[v.b]) * NB + v.c) * KB;
                scales = row_scales(sw, KB, v.k0);
            };
            bool more = walk.next(ahead);
            if (more) begin(ahead);
            while (more) {
                s = ahead;
                const int e = L.busy[s.b], first = L.start[e], n = L.start[e + 1] - first, ng = (n + 7) / 8;
                const float *now = sw;
                const float now_scales = scales;
                more = walk.next(ahead);
                if (more) begin(ahead);
                if (ok) {
                    float acc[8 * NG];
                    ok = sum_blocks<DOWN, NG>(a, ctl, acc, s, now, now_scales, KB, ng, taddr, it, b, bph);
                    if (ok) {
#pragma unroll
                        for (int m = 0; m < 8 * NG; ++m)
                            if (m < n) {
                                float *to = &ctl->sums[L.token[first + m]][row];
                                *to = fmaf(L.weight[first + m], acc[m], *to);
                            }
                    }
                }
                if (!s.end && more) continue;
                // the tile's end, or this CTA's.  A warp whose waits ran out comes here, too, so
                // that the others do not wait for it
                if (!named_bar_and(1, 128, ok)) break;
                const int64_t t0 = s.c * per, t1 = t0 + per;   // the tile's stages in the line
                const bool part = t0 < whole.pos || t1 > whole.end;
                // part: slot 1 of the CTA in which the tile starts, slot 0 of the others
                const int a0 = static_cast<int>(((t0 + 1) * G - 1) / all), a1 = static_cast<int>((t1 * G - 1) / all);
                const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (static_cast<int>(blockIdx.x) == a0 ? 1 : 0);
                // from here on a warp has a token's row, a lane four of its columns
                const int n0 = s.c * 128 + 4 * lane;
                float4 *sums = reinterpret_cast<float4 *>(&ctl->sums[0][4 * lane]);
                float4 *parts = reinterpret_cast<float4 *>(a.part + 4 * lane);
                for (int t = q; t < a.T; t += 4) {
                    const float4 v = sums[t * 32];
                    sums[t * 32] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (part) parts[(slot * a.T + t) * 32] = v;
                    else if (n0 < a.H) store_bf16x4(a.out + static_cast<int64_t>(t) * a.H + n0, v);
                }
                if (part) __threadfence();
                named_bar_sync(1, 128);
                if (!part) continue;
                if (row == 0) ctl->last = atomicAdd(&a.counters[a0], 1) == a1 - a0;
                named_bar_sync(1, 128);
                const bool last = ctl->last;
                named_bar_sync(1, 128);
                if (!last) continue;
                __threadfence();
                for (int t = q; t < a.T; t += 16) {   // four tokens at a time
                    float4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int i = a0; i <= a1; ++i) {
                        const float4 *from = parts + (static_cast<int64_t>(i) * 2 + (i == a0 ? 1 : 0)) * a.T * 32;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (t + 4 * k < a.T) {
                                const float4 w = __ldcg(from + (t + 4 * k) * 32);
                                v[k].x += w.x, v[k].y += w.y, v[k].z += w.z, v[k].w += w.w;
                            }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (t + 4 * k < a.T && n0 < a.H) store_bf16x4(a.out + static_cast<int64_t>(t + 4 * k) * a.H + n0, v[k]);
                }
            }
        }
    }

    if constexpr (DOWN) launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

}  // namespace bsfp8
