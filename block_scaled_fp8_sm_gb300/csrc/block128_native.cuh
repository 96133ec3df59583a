// block128_native.cuh -- the 128-granular product for power-of-two scales, on the
// block-scaled MMA (tcgen05 kind::mxf8f6f4): the scales are applied inside the tensor
// cores, so the sums stay in tensor memory over all of K and no partial is promoted.
//
// 128 x 256 tiles, persistent CTAs, rows of one product or of many experts (the tile
// order, loads and stores are block128_tile.cuh's).  The MMA takes one UE8M0 byte per row
// and 32 K; a 32-bit word per row holds the bytes of four 128-K blocks, and the four MMAs
// of a block all select the block's byte.  So one copy of 512 bytes (A: 32 lines of four
// rows' words) and two of 128 (B: eight equal lines, read four times) into tensor memory
// serve 512 K.
//
// Roles (384 threads): warp 0 producer, warp 1 MMA (one lane each), warps 2-3 scales:
// fp32 to exponent bytes, one entry of four K blocks at a time, up to four entries
// ahead; a scale that is not a positive normal power of two sets the status word.  Warps
// 4-11 read the sums once per tile, round them to bf16 and release the accumulator
// before they store.  Tensor memory: sums in columns 0-255, scales from column 256.
//
// 8192 x 28672 x 8192: 1125-1220 us (3150-3420 TFLOP/s, 82-89 % of twice the measured bf16
// rate) in runs of some ms, against 1360-1410 by promotion, and 1280-1320 in a loop of
// seconds, where power sets the clock, against 1530-1580.  Experts, runs of some ms: 16384
// rows over 16 of 4096 x 7168 338 us (promotion 374), 4001 skewed rows over 32 of 4104 x
// 2064 73 us (75).
#pragma once
#include "block128_tile.cuh"

namespace bsfp8 {

constexpr int N128_BN = 256;
constexpr int N128_SF_RING = 4;   // entries, in shared and in tensor memory (16 K blocks: more than the operand ring)
constexpr int N128_SF_A = 512, N128_SF_B = 128;                // bytes of lines: A's rows, one block of B
constexpr int N128_SF_ENTRY = N128_SF_A + 2 * N128_SF_B;
constexpr int N128_SF_COL0 = 256, N128_SF_COLS = 12;            // tensor memory: A 4 columns, B 4 per block

struct CtrlN128 : Ctrl128<N128_BN> {
    uint64_t sfull[N128_SF_RING], sempty[N128_SF_RING];
};

constexpr int smem_n128() {
    using C = Cfg128<N128_BN>;
    return 1024 + C::STAGES * (C::A_BYTES + C::B_BYTES) + C::STG + N128_SF_RING * N128_SF_ENTRY +
           static_cast<int>(sizeof(CtrlN128));
}

__device__ __forceinline__ bool is_pow2(float v) {
    const uint32_t b = __float_as_uint(v), e = b >> 23;   // a set sign makes e >= 256
    return (b & 0x007FFFFFu) == 0u && e != 0u && e < 255u;
}

__global__ void __launch_bounds__(T128_THREADS, 1) bsfp8_block128_native(const __grid_constant__ Tile128Args a) {
    using C = Cfg128<N128_BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_a = smem, *sm_b = smem + C::STAGES * C::A_BYTES;
    uint8_t *stg = sm_b + C::STAGES * C::B_BYTES;
    uint8_t *sf = stg + C::STG;
    CtrlN128 *ctl = reinterpret_cast<CtrlN128 *>(sf + N128_SF_RING * N128_SF_ENTRY);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int f = 0; f < N128_SF_RING; ++f) {
            mbar_init(&ctl->sfull[f], 2);
            mbar_init(&ctl->sempty[f], 1);
        }
        mbar_init(&ctl->tfull[0], 1);
        mbar_init(&ctl->tempty[0], T128_EPI_WARPS);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.tmA);
        tma_prefetch_desc(&a.tmA32);
        tma_prefetch_desc(&a.tmB);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    launch_dependents();
    wait_for_previous();
    if (warp == 2) count_tiles(a, ctl);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const int tiles = ctl->tiles, unit = static_cast<int>(blockIdx.x), units = static_cast<int>(gridDim.x);

    if (warp == 0) {
        if (elect_one()) {
            int it = 0, s = 0, withheld = -1;
            uint32_t ph = 1;
            bool ok = true;
            for (int t = unit; t < tiles && ok; t += units) {
                const Tile128 tt = tile128<N128_BN>(a, ctl, t);
                for (int kb = 0; kb < a.KB; ++kb) {
                    ok = wait128(&ctl->empty[s], ph, ctl, a);
                    if (!ok) break;
                    if (it == a.withhold && blockIdx.x == 0) withheld = s;
                    else load_stage<N128_BN>(a, &ctl->full[s], sm_a + s * C::A_BYTES, sm_b + s * C::B_BYTES, tt, kb);
                    ++it;
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // no load is in flight when the CTA leaves
            for (int d = max(0, it - C::STAGES); d < it; ++d) {
                if (d % C::STAGES == withheld) continue;
                const long long t0 = clock64();
                while (!mbar_try_wait(&ctl->full[d % C::STAGES], static_cast<uint32_t>(d / C::STAGES) & 1u))
                    if (clock64() - t0 > a.wait_limit) break;
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_mxf8f6f4(T128_BM, N128_BN, 0, 0);
            int s = 0, f = 0;
            uint32_t ph = 0, fph = 0, tph = 1;
            bool ok = true, ready = false;
            for (int t = unit; t < tiles && ok; t += units) {
                ok = wait128(&ctl->tempty[0], tph, ctl, a);
                if (!ok) break;
                tph ^= 1u;
                uint32_t sfa = 0;
                for (int kb = 0; kb < a.KB; ++kb) {
                    const uint32_t j = static_cast<uint32_t>(kb) & 3u;
                    if (j == 0) {
                        ok = wait128(&ctl->sfull[f], fph, ctl, a);
                        if (!ok) break;
                        tc_fence_after();
                        // the slot's last readers, the MMAs of four entries ago, are done:
                        // the stages loaded since then waited for them
                        sfa = tmem + N128_SF_COL0 + f * N128_SF_COLS;
                        const uint32_t lines = smem_u32(sf + f * N128_SF_ENTRY);
                        tmem_cp_32x128b_warpx4(sfa, sdesc_sf_lines32(lines));
                        tmem_cp_32x128b_warpx4(sfa + 4, sdesc_sf_lines(lines + N128_SF_A));
                        tmem_cp_32x128b_warpx4(sfa + 8, sdesc_sf_lines(lines + N128_SF_A + N128_SF_B));
                        mma_commit(&ctl->sempty[f]);
                        if (++f == N128_SF_RING) {
                            f = 0;
                            fph ^= 1u;
                        }
                    }
                    if (!ready) ok = wait128(&ctl->full[s], ph, ctl, a);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = sdesc_k_sw128(smem_u32(sm_a + s * C::A_BYTES));
                    const uint64_t bd = sdesc_k_sw128(smem_u32(sm_b + s * C::B_BYTES));
                    const uint32_t id = idesc | (j << 4) | (j << 29);
                    uint64_t *empty = &ctl->empty[s];
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // the next stage is looked for while the pipe is busy
                        if (i == 3) ready = mbar_test_wait(&ctl->full[s], ph);
                        mma_mxf8(tmem, ad + 2 * i, bd + 2 * i, id, sfa, sfa + 4, (kb | i) != 0);
                    }
                    mma_commit(empty);
                }
                if (!ok) break;
                mma_commit(&ctl->tfull[0]);
            }
            // all MMAs have completed before tensor memory is freed
            mma_commit(&ctl->drain);
            const long long t0 = clock64();
            while (!mbar_try_wait(&ctl->drain, 0))
                if (clock64() - t0 > a.wait_limit) break;
        }
    } else if (warp < 4) {
        // thread i writes the words of rows i and i + 64 (word w of line l: row 32 w + l)
        // and one word of B's lines
        const int i = (warp - 2) * 32 + lane;
        const bool vec = (a.KB & 3) == 0 && ((reinterpret_cast<uintptr_t>(a.sA) | reinterpret_cast<uintptr_t>(a.sB)) & 15) == 0;
        int f = 0;
        uint32_t fph = 1;
        bool ok = true, bad = false;
        for (int t = unit; t < tiles && ok; t += units) {
            const Tile128 tt = tile128<N128_BN>(a, ctl, t);
            const float *row[3];
            row[0] = a.sA + static_cast<int64_t>(min(tt.m0 + i, tt.hi - 1)) * a.KB;
            row[1] = a.sA + static_cast<int64_t>(min(tt.m0 + i + 64, tt.hi - 1)) * a.KB;
            row[2] = a.sB + (static_cast<int64_t>(tt.e) * a.NB + min(tt.n0 / 128 + (warp - 2), a.NB - 1)) * a.KB;
            for (int kb = 0; kb < a.KB; kb += 4) {
                uint32_t word[3];
#pragma unroll
                for (int r = 0; r < 3; ++r) {
                    float v[4];
                    if (vec) {
                        const float4 x = *reinterpret_cast<const float4 *>(row[r] + kb);
                        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = row[r][min(kb + j, a.KB - 1)];
                    }
                    word[r] = 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        bad |= !is_pow2(v[j]);
                        word[r] |= (__float_as_uint(v[j]) >> 23 & 0xFFu) << (8 * j);
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, wait128(&ctl->sempty[f], fph, ctl, a));
                if (!ok) break;
                uint32_t *lines = reinterpret_cast<uint32_t *>(sf + f * N128_SF_ENTRY);
                lines[lane * 4 + (warp - 2)] = word[0];
                lines[lane * 4 + (warp - 2) + 2] = word[1];
                lines[(N128_SF_A + (warp - 2) * N128_SF_B) / 4 + lane] = word[2];
                fence_proxy_async_smem();   // the lines become visible to tcgen05.cp
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->sfull[f]);
                if (++f == N128_SF_RING) {
                    f = 0;
                    fph ^= 1u;
                }
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(a.status, STATUS_SCALE);
    } else {
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * C::COLS;
        uint8_t *mine = stg + (warp - 4) * (32 * 64);
        uint32_t tph = 0;
        for (int t = unit; t < tiles; t += units) {
            const Tile128 tt = tile128<N128_BN>(a, ctl, t);
            if (!__all_sync(0xFFFFFFFFu, wait128(&ctl->tfull[0], tph, ctl, a))) break;
            tph ^= 1u;
            tc_fence_after();
            uint32_t w[C::COLS / 32][16];
#pragma unroll
            for (int x = 0; x < C::COLS / 32; ++x) {
                uint32_t p[2][16];
                tmem_ld_x16(taddr + 32 * x, p[0]);
                tmem_ld_x16(taddr + 32 * x + 16, p[1]);
                tmem_ld_wait_for(p[0]);
                tmem_ld_wait_for(p[1]);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    w[x][j] = bf16_pair(__uint_as_float(p[j >> 3][2 * (j & 7)]), __uint_as_float(p[j >> 3][2 * (j & 7) + 1]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[0]);
#pragma unroll
            for (int x = 0; x < C::COLS / 32; ++x) store_rows32(mine, a, tt, q, tt.n0 + h * C::COLS + 32 * x, w[x]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace bsfp8
