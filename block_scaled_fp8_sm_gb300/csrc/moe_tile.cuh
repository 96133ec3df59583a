// moe_tile.cuh -- the mixture-of-experts layer of moe_layer.cuh for more tokens or larger weights,
// on the tensor cores (tcgen05): the weights come by TMA and are never
// touched by a register.
//
// A weight tile's 256 rows are the M side of two MMAs, an expert's tokens their N side, in
// E4M3: a number v of the activations becomes two (x) or three (h) codes,
//   v / s = q0 + q1 / 32 + q2 / 1024,   each the nearest E4M3 of what the ones before leave,
// s the power of two that brings the largest of the token's 128 values of a K block to
// [2^7, 2^8).  Each code takes four of v's bits, so two hold the 8 bits of a bf16 exactly
// (down to 2^-14 of the block's largest; below, the error stays under 2^-22 of it), and
// three hold 12 bits of h.  The codes are columns of their own, and the epilogue adds
// (s_w s) (p0 + p1 / 32 + p2 / 1024) to fp32 registers for each 128-K block.
//
// The call is bound by the weights' bytes as long as every role keeps a K block (32 KB, 1430
// cycles of an SM's share of HBM) under that, each of them a chain of dependent instructions.
// 8 of 64 experts of 7168 x 2048: 16 tokens 352 us (6.9 TB/s), 32 tokens 409, 64 tokens 464 (6.1
// TB/s of 6.8: the makers' and the epilogue's 64 columns).  64 tokens before: mma.sync with the
// weights through registers 992, tiles of 128 rows 523 (an MMA costs ~60 cycles for its A side
// whatever N is, a TMA request ~70 of its thread), 256 481, an expert's K blocks walked without
// divisions 465, the parts of the cut tiles added by a kernel of their own 459.  Small weights pay
// the set-up: 19 tokens, 3 of 16 of 2064 x 1040 (98 MB) 32 us (27.7 with the weights in L2), of which
// 1.5 to 2 are the lists and 3 each change of kernels.
//
// NG (groups of eight tokens that the call has: 1, 2, 4, 8) sets the registers and the memory of
// the sums: with 8 for all of them 12 tokens, 2 of 16 of 2048 x 1024, take 27.8 us for 22.3.
//
// Roles (512 threads): warp 0 TMA, warp 1 MMA (one lane each), warps 4-11 epilogue (a thread
// owns a row of the tile and all tokens), six make the codes, four tokens of each eight of a K
// block in turn, so that the latency of their loads is spread over three blocks.
//
// Up: a tile is 128 columns of h, 16 gate rows and 16 up rows in turn, so that a warp holds
// both; CTAs take tiles in turn.  Down: a tile is 256 columns of the output with all busy
// experts one after the other, summed in shared memory; the K blocks of all tiles are one
// line, cut into equal pieces for the CTAs.  Where a cut goes through a tile, the parts go to
// the workspace and a third kernel adds them in order: no CTA waits for another, and calls repeat
// bit for bit.
//
// Every wait is bounded as in the other kernels.
#pragma once
#include "block128_tile.cuh"
#include "moe_layer.cuh"
#include "quant_math.cuh"

namespace bsfp8 {

constexpr int MT_THREADS = 512;
constexpr int MT_EPI_WARPS = 8;
constexpr int MT_CTAS = 152;           // one for each SM
constexpr int MT_ROWS = 256;           // weight rows of a tile
constexpr int MT_MAX_STAGES = 6;
constexpr int MT_MAX_BUFS = 4;
constexpr int MT_MAKERS = 6;           // warps that make codes
constexpr int MT_SX_RING = 16;         // slots of scales: the K blocks of all stages and partials, and more
constexpr int MT_SMEM = 232448;        // all that a CTA can have

// Four-dimensional tiled TMA load (coordinates innermost first).
__device__ __forceinline__ void tma_load_4d(const CUtensorMap *m, uint64_t *bar, void *dst, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

struct MoeTileArgs : MoeArgs {
    CUtensorMap tmW;
    float *part;              // [2 MT_CTAS][T][256]: sums of the tiles that a cut goes through,
    unsigned long long *has;  // [2 MT_CTAS] which tokens a part has: only their rows are there
    int *busy;                // how many experts have tokens
    uint32_t *status;
    long long wait_limit;
    int ring;                 // bytes of shared memory for the stages
    int withhold;             // test hook: CTA 0 never loads this stage (-1: off)
};

// DOWN, NG: groups of eight tokens that an expert can have.
template <bool DOWN>
constexpr int MT_PIECES = DOWN ? 3 : 2;
constexpr int MT_A_BYTES = MT_ROWS * 128;   // weights of a stage

template <bool DOWN, int NG>
struct CtrlMoe {
    uint64_t full[MT_MAX_STAGES], empty[MT_MAX_STAGES];   // full: the weights and the codes
    uint64_t tfull[MT_MAX_BUFS], tempty[MT_MAX_BUFS], drain;
    uint32_t tmem;
    int abort;
    alignas(16) float sx[MT_SX_RING][8 * NG];   // read four at a time
    alignas(16) float sums[DOWN ? 8 * NG : 1][MT_ROWS];
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

// A run of K blocks of one expert in one tile.
struct MoeSeg {
    int b, c, k0, k1;   // number of the busy expert, tile, K blocks [k0, k1)
    bool end;           // the tile's last
};

// The segments of this CTA in order; every role walks them alike.
template <bool DOWN>
struct MoeWalk {
    int64_t begin, end, all;   // up: tiles from here in steps of the grid; down: K blocks of the line
    int64_t left;              // down: K blocks not walked yet
    int ctas;                  // down: the CTAs that have some
    int busy, KB, tiles, b, c, k;

    __device__ __forceinline__ MoeWalk(int busy_, int KB_, int tiles_) : busy(busy_), KB(KB_), tiles(tiles_) {
        all = static_cast<int64_t>(tiles) * busy * (DOWN ? KB : 1);
        ctas = static_cast<int>(min(all, static_cast<int64_t>(gridDim.x)));
        const bool in = static_cast<int>(blockIdx.x) < ctas;
        begin = !in ? all : DOWN ? all * blockIdx.x / ctas : blockIdx.x;
        end = in && DOWN ? all * (blockIdx.x + 1) / ctas : all;
        left = DOWN ? end - begin : begin < all;
        b = c = k = 0;
        if (left > 0) {
            const int64_t tile = DOWN ? begin / KB : begin;   // tiles of experts: down expert by expert, up column by column
            k = DOWN ? static_cast<int>(begin - tile * KB) : 0;
            b = static_cast<int>(DOWN ? tile % busy : tile / tiles);
            c = static_cast<int>(DOWN ? tile / busy : tile % tiles);
        }
    }
    __device__ __forceinline__ bool next(MoeSeg &s) {
        if (left <= 0) return false;
        s.b = b;
        s.c = c;
        s.k0 = k;
        if constexpr (DOWN) {
            s.k1 = static_cast<int>(min(static_cast<int64_t>(KB), k + left));
            s.end = b + 1 == busy && s.k1 == KB;
            left -= s.k1 - k;
            k = 0;
            if (++b == busy) {
                b = 0;
                ++c;
            }
        } else {
            s.k1 = KB;
            s.end = true;
            c += gridDim.x;
            while (c >= tiles) {
                c -= tiles;
                ++b;
            }
            left = b < busy;
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

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Waits for the thread's tensor-memory loads; no use of p can be moved before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&p)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(p[0]), "+r"(p[1]), "+r"(p[2]), "+r"(p[3]), "+r"(p[4]), "+r"(p[5]), "+r"(p[6]), "+r"(p[7])
                 :
                 : "memory");
}

// Scales of the weights' K blocks kb .. kb + 15 of a tile, one in a lane of each half of a
// warp; sw: those of the thread's row, which are the same for a half.
__device__ __forceinline__ float row_scales(const float *sw, int KB, int kb) {
    return sw[min(kb + static_cast<int>(threadIdx.x & 15), KB - 1)];
}

__device__ __forceinline__ void store_bf16x4(__nv_bfloat16 *to, float4 v) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
}

// The epilogue's sum over the K blocks of a segment, ng groups of eight tokens.  next: the first
// scales; taddr, step: this half's columns of partial 0, and the columns of a partial.
template <bool DOWN, int NG, typename Ctl>
__device__ __forceinline__ bool sum_blocks(const MoeTileArgs &a, Ctl *ctl, float (&acc)[8 * NG], const MoeSeg &s,
                                           const float *sw, float next, int KB, int ng, uint32_t taddr, int step, int bufs,
                                           int &it, int &b, uint32_t &bph) {
#pragma unroll
    for (int j = 0; j < 8 * NG; ++j) acc[j] = 0.0f;
    const int lane = threadIdx.x & 31;
    float have = 0.0f;
    for (int kb = s.k0; kb < s.k1; ++kb) {
        const int in = (kb - s.k0) & 15;
        if (in == 0) {
            have = next;
            next = row_scales(sw, KB, kb + 16);
        }
        const float w = __shfl_sync(0xFFFFFFFFu, have, (lane & 16) + in);
        if (!__all_sync(0xFFFFFFFFu, wait_moe(&ctl->tfull[b], bph, ctl, a))) return false;
        tc_fence_after();
        const float4 *sx = reinterpret_cast<const float4 *>(ctl->sx[it % MT_SX_RING]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g < ng) {
                uint32_t p[16], r[8];   // the group's columns: eight for each code
                tmem_ld_x16(taddr + b * step + 8 * MT_PIECES<DOWN> * g, p);
                if constexpr (DOWN) tmem_ld_x8(taddr + b * step + 8 * MT_PIECES<DOWN> * g + 16, r);
                const float4 s0 = sx[2 * g], s1 = sx[2 * g + 1];
                const float f[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                tmem_ld_wait_for(p);
                if constexpr (DOWN) tmem_ld_wait_for(r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = __uint_as_float(p[8 + j]);
                    if constexpr (DOWN) v = fmaf(__uint_as_float(r[j]), 0.03125f, v);
                    acc[8 * g + j] = fmaf(w * f[j], fmaf(v, 0.03125f, __uint_as_float(p[j])), acc[8 * g + j]);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tempty[b]);
        ++it;
        if (++b == bufs) {
            b = 0;
            bph ^= 1u;
        }
    }
    return true;
}

template <bool DOWN, int NG>
__global__ void __launch_bounds__(MT_THREADS, 1) bsfp8_moe_tile(const __grid_constant__ MoeTileArgs a) {
    constexpr int PIECES = MT_PIECES<DOWN>;
    using Ctl = CtrlMoe<DOWN, NG>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + a.ring);
    const MoeLists L = moe_lists(smem + a.ring + moe_pad16(static_cast<int>(sizeof(Ctl))), a.T, a.top, a.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < MT_MAX_STAGES; ++s) {
            mbar_init(&ctl->full[s], 3);   // the weights, and the codes by two makers
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < MT_MAX_BUFS; ++b) {
            mbar_init(&ctl->tfull[b], 2);
            mbar_init(&ctl->tempty[b], MT_EPI_WARPS);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.tmW);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    // Down does not wait here: what it reads before its makers and epilogue wait (routing,
    // weights) is not written by the up kernel, and the kernels before that one had ended
    // when it let this one start.
    if constexpr (!DOWN) wait_for_previous();
    build_lists(a, L);
    if constexpr (!DOWN) launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    // a stage: a K block of the weights' 256 rows, and the codes of as many groups of eight
    // tokens as an expert has at most (the MMA takes an even number of eights); a partial: the
    // codes' columns, for the rows of each half
    const int busy = L.experts[0], most = (L.experts[1] + 7) / 8, eights = (PIECES * most + 1) / 2 * 2;
    const int stage_bytes = MT_A_BYTES + eights * 1024;
    const int stages = min(MT_MAX_STAGES, a.ring / stage_bytes);
    const int step = 16 * eights, bufs = min(MT_MAX_BUFS, 512 / max(step, 1));
    // Warps that make codes, half of a stage's each in turn.  Not more than all stages have
    // halves: a maker that looked further ahead would meet an `empty` barrier two rounds
    // behind, whose parity says that the stage is free.
    const int makers = min(MT_MAKERS, 2 * stages);
    const int K = DOWN ? a.I : a.H, KB = (K + 127) / 128;
    const int tiles = DOWN ? (a.H + MT_ROWS - 1) / MT_ROWS : (a.I + 127) / 128;
    MoeWalk<DOWN> walk(busy, KB, tiles);
    const MoeWalk<DOWN> whole = walk;
    MoeSeg s;

    if (warp == 0) {
        if (elect_one()) {
            int it = 0, st = 0, withheld = -1;
            uint32_t ph = 1;
            bool ok = true;
            while (ok && walk.next(s)) {
                const int e = L.busy[s.b];
                for (int kb = s.k0; kb < s.k1; ++kb) {
                    ok = wait_moe(&ctl->empty[st], ph, ctl, a);
                    if (!ok) break;
                    if (it == a.withhold && blockIdx.x == 0) {
                        withheld = it;
                    } else {
                        mbar_arrive_expect_tx(&ctl->full[st], MT_A_BYTES);
                        uint8_t *da = smem + st * stage_bytes;
                        if constexpr (DOWN) tma_load_2d(&a.tmW, &ctl->full[st], da, kb * 128, e * a.H + s.c * MT_ROWS);
                        else tma_load_4d(&a.tmW, &ctl->full[st], da, kb * 128, 0, 0, e * (a.I / 8) + s.c * 8);
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
                if (d == withheld) continue;
                while (!mbar_try_wait(&ctl->full[d % stages], static_cast<uint32_t>(d / stages) & 1u))
                    if (clock64() - t0 > a.wait_limit) break;
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            int st = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            bool ok = true;
            const uint64_t first = sdesc_k_sw128(smem_u32(smem));   // of the ring; an address adds its sixteenths
            const uint32_t next_stage = stage_bytes / 16;
            uint64_t ad = first;
            while (ok && walk.next(s)) {
                const int e = L.busy[s.b], ng = (L.start[e + 1] - L.start[e] + 7) / 8;
                const uint32_t idesc = idesc_f8f6f4(128, (PIECES * ng + 1) / 2 * 16);
                for (int kb = s.k0; kb < s.k1; ++kb) {
                    ok = wait_moe(&ctl->full[st], ph, ctl, a) && wait_moe(&ctl->tempty[b], bph, ctl, a);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + b * step;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_f8(d + h * (step / 2), ad + h * 1024 + 2 * i, ad + MT_A_BYTES / 16 + 2 * i, idesc, i > 0);
                    mma_commit(&ctl->tfull[b]);
                    mma_commit(&ctl->empty[st]);
                    mbar_arrive(&ctl->tfull[b]);   // the makers' scales are before this
                    ad += next_stage;
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                        ad = first;
                    }
                    if (++b == bufs) {
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
    } else if (warp < 4 || warp >= 12) {
        if constexpr (DOWN) wait_for_previous();
        // unit `it` is this warp's where it mod makers is its number: the first (it even) or last
        // four tokens of each group of eight of a stage.  Lane l makes the codes of the values
        // 4 l .. 4 l + 3 of each token; the next four tokens' are on their way meanwhile
        const int maker = warp < 4 ? warp - 2 : warp - 10;
        if (maker < makers) {
            int it = maker, st = maker / 2, unit = 0, end = 0, first = 0, n = 0;   // units [unit, end) of the segment are ahead
            uint32_t ph = 1;
            uint2 v[4];
            float hs[4];
            // `skip` units on, into the segments that follow
            auto advance = [&](int skip) {
                unit += skip;
                while (unit >= end) {
                    const int over = unit - end;
                    if (!walk.next(s)) return false;
                    unit = 2 * s.k0 + over;
                    end = 2 * s.k1;
                }
                const int e = L.busy[s.b];
                first = L.start[e];
                n = L.start[e + 1] - first;
                return true;
            };
            auto load = [&](int g) {
                const int k = unit / 2 * 128 + 4 * lane, m0 = 8 * g + 4 * (unit & 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = make_uint2(0u, 0u);
                    hs[i] = 0.0f;
                    if (m0 + i < n && k < K) {   // K is a multiple of 16
                        if constexpr (DOWN) {
                            const int64_t pair = L.pair[first + m0 + i];
                            v[i] = *reinterpret_cast<const uint2 *>(a.h + pair * a.I + k);
                            hs[i] = a.hs[pair * (a.I / 16) + k / 16];
                        } else {
                            v[i] = *reinterpret_cast<const uint2 *>(a.x + static_cast<int64_t>(L.token[first + m0 + i]) * a.H + k);
                        }
                    }
                }
            };
            bool more = advance(maker);
            if (more) load(0);
            while (more) {
                if (!__all_sync(0xFFFFFFFFu, wait_moe(&ctl->empty[st], ph, ctl, a))) break;
                const int r = 4 * (it & 1), ng = (n - r + 7) / 8;   // groups that have tokens of this half
                uint8_t *db = smem + st * stage_bytes + MT_A_BYTES + r * 128;
                float *sx = ctl->sx[(it >> 1) % MT_SX_RING] + r;
                if (ng == 0) {
                    more = advance(makers);
                    if (more) load(0);
                }
                for (int g = 0; g < ng; ++g) {
                    // fp16 with the block's largest in [2^7, 2^8): sixteen values of h go to 0 below 2^-24 of it,
                    // and fp16's own smallest step is 2^-31 of it
                    __half2 f[4][2];
                    float inverse[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (DOWN) {   // h's own scales (of the largest of 16 in [2^7, 2^8)) say enough
                            const float top = fmaxf(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(hs[i]))), 0x1p-126f);
                            const __half2 k = __float2half2_rn(hs[i] * __uint_as_float((254u << 23) - __float_as_uint(top)));
                            f[i][0] = __hmul2(*reinterpret_cast<const __half2 *>(&v[i].x), k);
                            f[i][1] = __hmul2(*reinterpret_cast<const __half2 *>(&v[i].y), k);
                            inverse[i] = top < 0x1p121f ? top : INFINITY;   // 2^121: of an infinite h
                        } else {
                            uint32_t a0, a1;
                            asm("abs.bf16x2 %0, %1;" : "=r"(a0) : "r"(v[i].x));
                            asm("abs.bf16x2 %0, %1;" : "=r"(a1) : "r"(v[i].y));
                            asm("max.bf16x2 %0, %0, %1;" : "+r"(a0) : "r"(a1));
                            const uint32_t top = max(a0 << 16, a0 & 0xFFFF0000u);
                            const float sc = scale_to_e4m3(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top)), inverse[i]);
                            f[i][0] = __floats2half2_rn(bf16_lo(v[i].x) * sc, bf16_hi(v[i].x) * sc);
                            f[i][1] = __floats2half2_rn(bf16_lo(v[i].y) * sc, bf16_hi(v[i].y) * sc);
                        }
                    }
                    if (lane == 0)
                        *reinterpret_cast<float4 *>(sx + 8 * g) = make_float4(inverse[0], inverse[1], inverse[2], inverse[3]);
                    if (g + 1 < ng) {
                        load(g + 1);
                    } else {
                        more = advance(makers);
                        if (more) load(0);
                    }
#pragma unroll
                    for (int p = 0; p < PIECES; ++p)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            // 16-byte pieces are exchanged by the row's low bits
                            *reinterpret_cast<uint32_t *>(db + (g * PIECES + p) * 1024 + i * 128 +
                                                          ((((lane >> 2) ^ (r + i)) << 4) | ((lane & 3) << 2))) = take_codes(f[i]);
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
    } else {
        if constexpr (DOWN) wait_for_previous();
        const int q = warp & 3, half = (warp - 4) >> 2, row = half * 128 + q * 32 + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * (step / 2);
        int it = 0, b = 0;
        uint32_t bph = 0;
        bool ok = true;
        if constexpr (!DOWN) {
            const int NB = (2 * a.I + 127) / 128;
            const float *sw = a.s1;
            float scales = 0.0f;
            auto begin = [&](const MoeSeg &v) {   // a segment's first scales
                const int col = min(v.c * 128 + half * 64 + q * 16 + (lane & 15), a.I - 1);
                sw = a.s1 + (static_cast<int64_t>(L.busy[v.b]) * NB + ((lane < 16 ? 0 : a.I) + col) / 128) * KB;
                scales = row_scales(sw, KB, v.k0);
            };
            bool more = walk.next(s);
            if (more) begin(s);
            while (ok && more) {
                const int e = L.busy[s.b], first = L.start[e], n = L.start[e + 1] - first, ng = (n + 7) / 8;
                const int col = s.c * 128 + half * 64 + q * 16 + (lane & 15);   // lanes 0-15 hold its gate, 16-31 its up
                float acc[8 * NG];
                ok = sum_blocks<DOWN, NG>(a, ctl, acc, s, sw, scales, KB, ng, taddr, step, bufs, it, b, bph);
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
                            const float sc = scale_to_half<7>(amax, inverse);   // as the codes are made from
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
            const int64_t per = static_cast<int64_t>(busy) * KB, all = walk.all, G = walk.ctas;
            const int NB = (a.H + 127) / 128;
            if (busy == 0)   // no token has an expert
                for (int c = blockIdx.x; c < tiles; c += gridDim.x)
                    for (int t = 0; t < a.T; ++t)
                        if (c * MT_ROWS + row < a.H)
                            a.out[static_cast<int64_t>(t) * a.H + c * MT_ROWS + row] = __float2bfloat16_rn(0.0f);
            if (blockIdx.x == 0 && row == 0) *a.busy = busy;
            for (int t = 0; t < a.T; ++t) ctl->sums[t][row] = 0.0f;
            unsigned long long touched = 0ull;   // tokens that the sums hold something of
            MoeSeg ahead;   // the next segment, whose first scales are on their way
            const float *sw = a.s2;
            float scales = 0.0f;
            auto begin = [&](const MoeSeg &v) {
                sw = a.s2 + (static_cast<int64_t>(L.busy[v.b]) * NB + min(2 * v.c + half, NB - 1)) * KB;
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
                    ok = sum_blocks<DOWN, NG>(a, ctl, acc, s, now, now_scales, KB, ng, taddr, step, bufs, it, b, bph);
                    if (ok) {   // four tokens at a time: they are different ones
#pragma unroll
                        for (int m = 0; m < 8 * NG; m += 4) {
                            if (m >= n) break;
                            float *to[4], v[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int at = first + min(m + i, n - 1);
                                to[i] = &ctl->sums[L.token[at]][row];
                                v[i] = fmaf(L.weight[at], acc[m + i], *to[i]);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (m + i < n) *to[i] = v[i];
                        }
                    }
                }
                for (int m = lane; m < n; m += 32) touched |= 1ull << L.token[first + m];
                if (!s.end && more) continue;
                // the tile's end, or this CTA's.  A warp whose waits ran out comes here, too, so
                // that the others do not wait for it
                if (!named_bar_and(1, 256, ok)) break;
                const int64_t t0 = s.c * per, t1 = t0 + per;   // the tile's K blocks in the line
                const bool part = t0 < whole.begin || t1 > whole.end;
                // part: slot 1 of the CTA in which the tile starts, slot 0 of the others
                const int a0 = static_cast<int>(((t0 + 1) * G - 1) / all);
                const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (static_cast<int>(blockIdx.x) == a0 ? 1 : 0);
                // from here on a warp has a token's row, a lane eight of its columns (four and four)
                const unsigned long long tokens =
                    static_cast<unsigned long long>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(touched >> 32))) << 32 |
                    __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(touched));
                touched = 0ull;
                const int n0 = s.c * MT_ROWS + 4 * lane;
                float4 *sums = reinterpret_cast<float4 *>(&ctl->sums[0][4 * lane]);
                float4 *parts = reinterpret_cast<float4 *>(a.part + 4 * lane);
                constexpr int LD = MT_ROWS / 4;   // 16-byte pieces of a row
                for (int t = warp - 4; t < a.T; t += MT_EPI_WARPS) {
                    const bool there = tokens >> t & 1ull;
                    if (part && !there) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 v = sums[t * LD + 32 * h];
                        if (there) sums[t * LD + 32 * h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (part) parts[(slot * a.T + t) * LD + 32 * h] = v;
                        else if (n0 + 128 * h < a.H) store_bf16x4(a.out + static_cast<int64_t>(t) * a.H + n0 + 128 * h, v);
                    }
                }
                if (part && warp == 4 && lane == 0) a.has[slot] = tokens;
                named_bar_sync(1, 256);   // the sums are zeros again
            }
        }
    }

    if constexpr (DOWN) launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The tiles that a cut goes through: a CTA adds the parts of one token and one tile in their
// order, eight on their way, four columns a thread.  A kernel of its own, because it is all latency:
// by the CTA that came last to a tile, the layer took 34.7 us for 28.6 (44 tokens, 2 of 9 experts of
// 1376 x 1584, 6 tiles of 25 parts, weights in L2), 32.1 for 26.8 (19 tokens, 3 of 16 of 2064 x 1040,
// in L2) and 468 for 459 (64 tokens, 8 of 64 of 7168 x 2048).
constexpr int MT_JOIN_THREADS = MT_ROWS / 4;

__global__ void __launch_bounds__(MT_JOIN_THREADS) bsfp8_moe_join(const MoeTileArgs a) {
    const int c = blockIdx.x, t = blockIdx.y, n = c * MT_ROWS + 4 * static_cast<int>(threadIdx.x);
    wait_for_previous();
    launch_dependents();
    // the cuts of MoeWalk<true>
    const int64_t per = static_cast<int64_t>(*a.busy) * ((a.I + 127) / 128), all = per * gridDim.x;
    if (all == 0) return;
    const int64_t G = min(all, static_cast<int64_t>(MT_CTAS)), t0 = c * per, t1 = t0 + per;
    const int a0 = static_cast<int>(((t0 + 1) * G - 1) / all), a1 = static_cast<int>((t1 * G - 1) / all);
    if (a0 == a1) return;   // the tile is one CTA's
    const float4 *parts = reinterpret_cast<const float4 *>(a.part) + threadIdx.x;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = a0; i0 <= a1; i0 += 32) {
        const int i = i0 + static_cast<int>(threadIdx.x & 31);
        uint32_t left = __ballot_sync(0xFFFFFFFFu, i <= a1 && (a.has[2 * min(i, a1) + (i == a0 ? 1 : 0)] >> t & 1ull));
        while (left) {
            float4 w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int from = i0 + __ffs(left) - 1;
                w[x] = left ? parts[((static_cast<int64_t>(from) * 2 + (from == a0 ? 1 : 0)) * a.T + t) * MT_JOIN_THREADS]
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                left &= left - 1u;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) v.x += w[x].x, v.y += w[x].y, v.z += w[x].z, v.w += w[x].w;
        }
    }
    if (n < a.H) store_bf16x4(a.out + static_cast<int64_t>(t) * a.H + n, v);
}

}  // namespace bsfp8
