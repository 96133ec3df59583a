// block128_tile.cuh -- the 128-granular product on the tensor cores (tcgen05,
// tensor-memory partials, TMA operands), for one product or for the ragged rows
// of many experts.
//
//   C[m,n] = bf16( sum_kb sA[m][kb] sB[n/128][kb] sum_{k in kb} A[m,k] B[n,k] )
//
// The inner sum of a 128-K block is four unscaled kind::f8f6f4 MMAs (K = 32) into
// one tensor-memory partial.  The epilogue warps add it to fp32 registers:
// acc = fma(s, partial, acc).  A thread owns one row of the tile and columns of one
// 128-column block of B, so s = sA[m][kb] sB[nb][kb] is one number per thread and
// block, and 128 K values cost one FMA per output.
//
// Roles (384 threads): warp 0 producer (one lane: one TMA box per operand and 128-K
// stage, 128-byte swizzle); warp 1 MMA (one lane); warps 4-11 epilogue: warp w reads
// the tensor-memory lanes (rows) 32 (w mod 4) .., columns of half (w - 4) / 4.  The
// partials are double- (BN = 256) or quadruple-buffered (BN = 128).
//
// What bounds it: a partial's round trip.  The four MMAs of a block keep the tensor pipe
// busy ~505 cycles, the epilogue needs ~660 for its eight load-and-FMA pieces and the
// hand-over, and with two 256-column partials the sum of both and of the two signals is
// paid every second block: ~870 cycles a block, the tensor pipe 55-66 % busy (4096^3 61 us
// alone, 65 in a loop of seconds; 8192 x 28672 x 8192 1360-1410 us, 2730-2830 TFLOP/s, in
// runs of some ms, 1530-1580, 2440-2520, in such a loop, where power holds the clock near
// 1.8 GHz).  Measured alone, and slower: more, narrower partials (128 columns 72 us: an N = 128 MMA
// costs as much as N = 256), 192 columns with twelve epilogue warps (71), sixteen warps
// (78), packed FMAs (67: the loaded values have to be moved into pairs), two pieces in
// flight (61-70), scales staged in shared memory by the idle warps (73).  The role threads
// are chosen by elect.sync: with lane == 0 the MMA thread's own loop took 20 % longer.
//
// Without SPLIT a CTA is persistent over tiles; with SPLIT a cluster of CTAs shares
// one tile, each taking a range of K blocks: the partial sums meet in the CTAs' own
// shared memory and are added in rank order over distributed shared memory, so a
// call repeats bit for bit.
//
// Every wait is bounded as in the other kernels: on expiry the status word is set,
// the roles leave, loads and MMAs in flight are drained and the kernel returns.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "block128_rows.cuh"
#include "ptx.cuh"

namespace bsfp8 {

constexpr int T128_BM = 128;
constexpr int T128_THREADS = 384;
constexpr int T128_EPI_WARPS = 8;
constexpr int T128_MAX_EXPERTS = 1024;
constexpr int T128_MAX_SPLIT = 4;   // CTAs of a cluster
// Registers per thread after the split: the launch holds 384 x 168 = 64512; the role
// warpgroup keeps 80, the two epilogue warpgroups take 208 (128 x 80 + 256 x 208 =
// 63488): a thread holds 128 sums and 16 values of a partial.  At 168 the K loop spilled:
// 4096^3 109 us, with the split 70 us.
constexpr int T128_ROLE_REGS = 80;
constexpr int T128_EPI_REGS = 208;

struct Tile128Args {
    // A in boxes of 128 rows, and of 32 for tiles of up to 64 rows: what such a tile does
    // not have is not fetched (those rows of the slot keep old bytes, which feed only
    // sums that are never stored); more boxes would cost more requests than one of 128.
    CUtensorMap tmA, tmA32, tmB;
    const float *sA, *sB;
    __nv_bfloat16 *C;
    const int32_t *offsets;   // [E + 1], or null: one product
    uint32_t *status;
    long long wait_limit;
    int M, N, KB, NB, E, mt, nt;
    int group;                // m-tiles whose A stays in L2 while B passes once
    int withhold;             // test hook: CTA 0 never loads this stage (-1: off)
};

template <int BN>
struct Cfg128 {
    static constexpr int A_BYTES = T128_BM * 128;
    static constexpr int B_BYTES = BN * 128;
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr int BUFS = 512 / BN;
    static constexpr int COLS = BN / 2;   // columns per epilogue thread
    static constexpr int STG = T128_EPI_WARPS * 32 * 64;   // 32 rows x 32 bf16 columns per epilogue warp
};

template <int BN>
struct Ctrl128 {
    uint64_t full[Cfg128<BN>::STAGES], empty[Cfg128<BN>::STAGES];
    uint64_t tfull[Cfg128<BN>::BUFS], tempty[Cfg128<BN>::BUFS], drain;
    uint32_t tmem;
    int abort, tiles;
    int start[T128_MAX_EXPERTS + 1];   // experts: first tile of each,
    int2 rows[T128_MAX_EXPERTS];       // and its rows
};

template <int BN>
constexpr int smem128() {
    return 1024 + Cfg128<BN>::STAGES * (Cfg128<BN>::A_BYTES + Cfg128<BN>::B_BYTES) + Cfg128<BN>::STG +
           static_cast<int>(sizeof(Ctrl128<BN>));
}

// Bounded wait: polls, and looks at the clock and the abort flag every 16 polls.
template <typename Ctl>
__device__ __forceinline__ bool wait128(uint64_t *bar, uint32_t parity, Ctl *ctl, const Tile128Args &a) {
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

// Waits for this thread's tensor-memory loads; p passes through it, so that no use of p
// can be moved before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&p)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(p[0]), "+r"(p[1]), "+r"(p[2]), "+r"(p[3]), "+r"(p[4]), "+r"(p[5]), "+r"(p[6]), "+r"(p[7]),
                   "+r"(p[8]), "+r"(p[9]), "+r"(p[10]), "+r"(p[11]), "+r"(p[12]), "+r"(p[13]), "+r"(p[14]), "+r"(p[15])
                 :
                 : "memory");
}

struct Tile128 {
    int m0, hi, n0, e;   // first row, end of its rows, first column, expert
};

// Tile t of the launch: experts in order, or groups of a.group m-tiles; m fastest.
template <int BN, typename Ctl>
__device__ __forceinline__ Tile128 tile128(const Tile128Args &a, const Ctl *ctl, int t) {
    Tile128 r;
    if (a.offsets) {
        int e0 = 0, e1 = a.E;   // start[e0] <= t < start[e1]
        while (e1 - e0 > 1) {
            const int mid = (e0 + e1) >> 1;
            if (ctl->start[mid] <= t) e0 = mid;
            else e1 = mid;
        }
        const int2 rows = ctl->rows[e0];
        const int in = t - ctl->start[e0], mt = (rows.y - rows.x + T128_BM - 1) / T128_BM;
        r.e = e0;
        r.hi = rows.y;
        r.m0 = rows.x + (in % mt) * T128_BM;
        r.n0 = in / mt * BN;
    } else {
        const int per = a.group * a.nt, grp = t / per, first = grp * a.group;
        const int size = min(a.mt - first, a.group), in = t - grp * per;
        r.e = 0;
        r.m0 = (first + in % size) * T128_BM;
        r.n0 = in / size * BN;
        r.hi = a.M;
    }
    return r;
}

template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of a converged warp.  The role of a single thread is chosen this way and not
// by lane == 0: the compiler then knows that one thread runs it, and issues the tcgen05
// and TMA instructions without a loop over the active lanes.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

// 16 bytes at this shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank));
    return v;
}

// acc += s * (16 columns of a partial): the load, its wait and the FMAs as one block, so
// that the compiler keeps this order whatever surrounds it (loads hoisted over the FMAs of
// the piece before, or two pieces in flight, ran slower: the other warp of the
// sub-partition fills the wait).
__device__ __forceinline__ void promote16(float *acc, uint32_t taddr, float s) {
    asm volatile(
        "{\n\t.reg .b32 p0, p1, p2, p3, p4, p5, p6, p7, p8, p9, p10, p11, p12, p13, p14, p15;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {p0,p1,p2,p3,p4,p5,p6,p7,p8,p9,p10,p11,p12,p13,p14,p15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "fma.rn.f32 %0, p0, %17, %0;\n\t"
        "fma.rn.f32 %1, p1, %17, %1;\n\t"
        "fma.rn.f32 %2, p2, %17, %2;\n\t"
        "fma.rn.f32 %3, p3, %17, %3;\n\t"
        "fma.rn.f32 %4, p4, %17, %4;\n\t"
        "fma.rn.f32 %5, p5, %17, %5;\n\t"
        "fma.rn.f32 %6, p6, %17, %6;\n\t"
        "fma.rn.f32 %7, p7, %17, %7;\n\t"
        "fma.rn.f32 %8, p8, %17, %8;\n\t"
        "fma.rn.f32 %9, p9, %17, %9;\n\t"
        "fma.rn.f32 %10, p10, %17, %10;\n\t"
        "fma.rn.f32 %11, p11, %17, %11;\n\t"
        "fma.rn.f32 %12, p12, %17, %12;\n\t"
        "fma.rn.f32 %13, p13, %17, %13;\n\t"
        "fma.rn.f32 %14, p14, %17, %14;\n\t"
        "fma.rn.f32 %15, p15, %17, %15;\n\t"
        "}"
        : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3]),
          "+f"(acc[4]), "+f"(acc[5]), "+f"(acc[6]), "+f"(acc[7]),
          "+f"(acc[8]), "+f"(acc[9]), "+f"(acc[10]), "+f"(acc[11]),
          "+f"(acc[12]), "+f"(acc[13]), "+f"(acc[14]), "+f"(acc[15])
        : "r"(taddr), "f"(s)
        : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 32 bf16 columns (16 words) of each lane's row to C, through the warp's 2 KB of staging:
// eight rows of 64 contiguous bytes per store.  16-byte pieces are exchanged so that the
// rows of a quarter-warp hit different banks.  q: the warp's quarter of the tile's rows.
__device__ __forceinline__ void store_rows32(uint8_t *mine, const Tile128Args &a, const Tile128 &tt, int q, int col,
                                             const uint32_t (&w)[16]) {
    const int lane = threadIdx.x & 31;
    uint4 *row = reinterpret_cast<uint4 *>(mine + lane * 64);
#pragma unroll
    for (int c = 0; c < 4; ++c)
        row[c ^ ((lane >> 1) & 3)] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int rr = i * 8 + (lane >> 2), c = lane & 3;
        const uint4 v = *reinterpret_cast<const uint4 *>(mine + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
        const int mm = tt.m0 + q * 32 + rr;
        if (mm < tt.hi && col + 8 * c < a.N)
            *reinterpret_cast<uint4 *>(a.C + static_cast<int64_t>(mm) * a.N + col + 8 * c) = v;
    }
    __syncwarp();
}

// First tile of each expert (a running sum over one warp), or the tile count of one
// product.  Reports an offset table that decreases or leaves [0, M].
template <typename Ctl>
__device__ __forceinline__ void count_tiles(const Tile128Args &a, Ctl *ctl) {
    const int lane = threadIdx.x & 31;
    if (!a.offsets) {
        if (lane == 0) ctl->tiles = a.mt * a.nt;
        return;
    }
    int base = 0, top = 0;   // tiles so far; the rows below `top` have an expert
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < a.E) {
            expert_rows(a.offsets, e, a.M, lo, hi);
            if (blockIdx.x == 0 && (lo != a.offsets[e] || hi != a.offsets[e + 1] || hi < lo))
                atomicOr(a.status, STATUS_RECORD);
        }
        // ranges that overlap (a bad table) are cut, so that there are never more tiles
        // than a table of ascending rows can have
        int most = hi;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, most, o);
            if (lane >= o) most = max(most, v);
        }
        const int before = __shfl_up_sync(0xFFFFFFFFu, most, 1);
        lo = max(lo, lane > 0 ? max(before, top) : top);
        top = max(top, __shfl_sync(0xFFFFFFFFu, most, 31));
        const int n = hi > lo ? (hi - lo + T128_BM - 1) / T128_BM * a.nt : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        if (e < a.E) {
            ctl->start[e] = base + sum - n;
            ctl->rows[e] = make_int2(lo, hi);
        }
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) ctl->start[a.E] = ctl->tiles = base;
}

// The producer's loads of one 128-K stage (see Tile128Args: boxes of A).
template <int BN>
__device__ __forceinline__ void load_stage(const Tile128Args &a, uint64_t *full, uint8_t *da, uint8_t *db,
                                           const Tile128 &tt, int kb) {
    using C = Cfg128<BN>;
    const int rows = tt.hi - tt.m0, small = rows <= 64 ? (rows + 31) / 32 : 0;
    mbar_arrive_expect_tx(full, (small ? small * 4096 : C::A_BYTES) + C::B_BYTES);
    if (small == 0) tma_load_2d(&a.tmA, full, da, kb * 128, tt.m0);
    for (int i = 0; i < small; ++i) tma_load_2d(&a.tmA32, full, da + i * 4096, kb * 128, tt.m0 + i * 32);
    tma_load_2d(&a.tmB, full, db, kb * 128, tt.e * a.N + tt.n0);
}

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(T128_THREADS, 1) bsfp8_block128_tile(const __grid_constant__ Tile128Args a) {
    using C = Cfg128<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_a = smem, *sm_b = smem + C::STAGES * C::A_BYTES;
    uint8_t *stg = sm_b + C::STAGES * C::B_BYTES;
    Ctrl128<BN> *ctl = reinterpret_cast<Ctrl128<BN> *>(stg + C::STG);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank = 0, ranks = 1;
    if constexpr (SPLIT) {
        rank = cluster_ctarank();
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < C::BUFS; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], T128_EPI_WARPS);
        }
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
    if (warp == 2) {
        count_tiles(a, ctl);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const int tiles = ctl->tiles;
    const int unit = static_cast<int>(blockIdx.x / ranks), units = static_cast<int>(gridDim.x / ranks);
    const int kb0 = static_cast<int>(static_cast<int64_t>(a.KB) * rank / ranks);
    const int kb1 = static_cast<int>(static_cast<int64_t>(a.KB) * (rank + 1) / ranks);

    if (warp < 4) {
        setmaxnreg_dec<T128_ROLE_REGS>();
        if (warp == 0) {
            if (elect_one()) {
                int it = 0, s = 0, withheld = -1;
                uint32_t ph = 1;
                bool ok = true;
                for (int t = unit; t < tiles && ok; t += units) {
                    const Tile128 tt = tile128<BN>(a, ctl, t);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        ok = wait128(&ctl->empty[s], ph, ctl, a);
                        if (!ok) break;
                        if (it == a.withhold && blockIdx.x == 0) {
                            withheld = s;
                        } else {
                            load_stage<BN>(a, &ctl->full[s], sm_a + s * C::A_BYTES, sm_b + s * C::B_BYTES, tt, kb);
                        }
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
                constexpr uint32_t idesc = idesc_f8f6f4(T128_BM, BN);
                int s = 0, b = 0;
                uint32_t ph = 0, bph = 1;
                bool ok = true;
                for (int t = unit; t < tiles && ok; t += units) {
                    for (int kb = kb0; kb < kb1; ++kb) {
                        const uint64_t ad = sdesc_k_sw128(smem_u32(sm_a + s * C::A_BYTES));
                        const uint64_t bd = sdesc_k_sw128(smem_u32(sm_b + s * C::B_BYTES));
                        // the operands first: the partial's release is what comes last
                        ok = wait128(&ctl->full[s], ph, ctl, a) && wait128(&ctl->tempty[b], bph, ctl, a);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_f8(tmem + b * BN, ad + 2 * i, bd + 2 * i, idesc, i > 0);
                        mma_commit(&ctl->tfull[b]);
                        mma_commit(&ctl->empty[s]);
                        if (++s == C::STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
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
        }
    } else {
        setmaxnreg_inc<T128_EPI_REGS>();
        const int q = warp & 3, h = (warp - 4) >> 2;
        const int r = q * 32 + lane;   // row of the tile
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * C::COLS;
        uint8_t *mine = stg + (warp - 4) * (32 * 64);
        int b = 0;
        uint32_t bph = 0;
        bool ok = true;
        // a tile's place, its scales' addresses and the first two of them
        Tile128 tt{};
        const float *psa = nullptr, *psb = nullptr;
        float sa = 0.0f, sb = 0.0f;
        auto begin = [&](int t) {
            tt = tile128<BN>(a, ctl, t);
            const int m = min(tt.m0 + r, tt.hi - 1);
            const int nb = min((tt.n0 + h * C::COLS) / 128, a.NB - 1);
            psa = a.sA + static_cast<int64_t>(m) * a.KB;
            psb = a.sB + (static_cast<int64_t>(tt.e) * a.NB + nb) * a.KB;
            if (kb0 < kb1) {
                sa = psa[kb0];
                sb = psb[kb0];
            }
        };
        if (unit < tiles) begin(unit);
        for (int t = unit; t < tiles && ok; t += units) {
            float acc[C::COLS];
#pragma unroll
            for (int j = 0; j < C::COLS; ++j) acc[j] = 0.0f;
            for (int kb = kb0; kb < kb1; ++kb) {
                const float sc = sa * sb;
                const int next = min(kb + 1, kb1 - 1);
                sa = psa[next];
                sb = psb[next];
                ok = __all_sync(0xFFFFFFFFu, wait128(&ctl->tfull[b], bph, ctl, a));
                if (!ok) break;
                tc_fence_after();
                constexpr int PIECES = C::COLS / 16;
#pragma unroll
                for (int x = 0; x + 1 < PIECES; ++x) promote16(acc + 16 * x, taddr + b * BN + 16 * x, sc);
                uint32_t p[16];
                tmem_ld_x16(taddr + b * BN + 16 * (PIECES - 1), p);
                tmem_ld_wait_for(p);
                tc_fence_before();   // the partial is in registers
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->tempty[b]);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    acc[C::COLS - 16 + j] = fmaf(__uint_as_float(p[j]), sc, acc[C::COLS - 16 + j]);
                if (++b == C::BUFS) {
                    b = 0;
                    bph ^= 1u;
                }
            }
            if (!ok) break;
            const Tile128 cur = tt;
            // the next tile's first scales are on their way while this one is stored
            if (t + units < tiles) begin(t + units);
            if constexpr (SPLIT) {
                // the partial sums go to the operand ring's memory (nothing is in
                // flight there any more: the last partial came after the last load),
                // 16-byte pieces exchanged by row so that the eight rows of a
                // quarter-warp hit different banks
                float4 *red = reinterpret_cast<float4 *>(smem);
#pragma unroll
                for (int j = 0; j < C::COLS / 4; ++j)
                    red[r * (BN / 4) + ((h * (C::COLS / 4) + j) ^ (r & 7))] =
                        make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
            } else {
#pragma unroll
                for (int x = 0; x < C::COLS / 32; ++x) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = bf16_pair(acc[32 * x + 2 * j], acc[32 * x + 2 * j + 1]);
                    store_rows32(mine, a, cur, q, cur.n0 + h * C::COLS + 32 * x, w);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (SPLIT) {
        cluster_sync();   // every CTA's partial sums are in its shared memory
        if (unit < tiles) {
            const Tile128 tt = tile128<BN>(a, ctl, unit);
            const uint32_t base = smem_u32(smem);
            // the rows that exist, four columns a thread, shared out evenly; all
            // ranks' pieces are in flight before the first is added
            const int pieces = min(T128_BM, tt.hi - tt.m0) * (BN / 4);
            const int per = (pieces + static_cast<int>(ranks) - 1) / static_cast<int>(ranks);
            const int end = min(pieces, (static_cast<int>(rank) + 1) * per);
            for (int i = static_cast<int>(rank) * per + threadIdx.x; i < end; i += T128_THREADS) {
                const int r = i / (BN / 4), c = i % (BN / 4);
                const uint32_t off = static_cast<uint32_t>(r * (BN / 4) + (c ^ (r & 7))) * 16u;
                float4 v[T128_MAX_SPLIT];
#pragma unroll
                for (uint32_t k = 0; k < T128_MAX_SPLIT; ++k)
                    v[k] = k < ranks ? ld_dsmem_f32x4(base + off, k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (uint32_t k = 1; k < T128_MAX_SPLIT; ++k) {
                    v[0].x += v[k].x;
                    v[0].y += v[k].y;
                    v[0].z += v[k].z;
                    v[0].w += v[k].w;
                }
                const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0].x, v[0].y), hi = __floats2bfloat162_rn(v[0].z, v[0].w);
                if (tt.n0 + 4 * c < a.N)
                    *reinterpret_cast<uint2 *>(a.C + static_cast<int64_t>(tt.m0 + r) * a.N + tt.n0 + 4 * c) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            }
        }
        cluster_sync();   // no CTA leaves while a peer reads its shared memory
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace bsfp8
