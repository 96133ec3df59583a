"""GPU parity of the 128-granular product and its expert-grouped form with a
plain 64-bit product, within the acceptance bound of the other GEMM calls
(bf16 rounding 2^-9 relative, and 1e-5 of the magnitude sum for the fp32
accumulation)."""
import itertools

import numpy as np
import pytest
import torch

from tests._accept import bf16_to_f64, check
from tests._block128 import Product, product

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bs():
    import block_scaled_fp8_sm_gb300 as mod
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    mod.library()
    return mod


def _guarded(M, N):
    """C with a row before and a row after it that must not be written."""
    whole = torch.full((M + 2, N), -7.0, dtype=torch.bfloat16, device=DEV)
    return whole, whole[1:M + 1]


SHAPES = [
    (1, 8, 16), (1, 4096, 7168), (2, 136, 144), (7, 24, 128), (8, 128, 256), (9, 256, 1040), (16, 264, 400),
    (31, 512, 512), (33, 1000, 272), (64, 256, 4096), (65, 128, 2064), (127, 8, 1024), (128, 384, 128), (129, 264, 1168),
    (200, 520, 640), (257, 1288, 912), (384, 256, 2048), (1000, 776, 528), (2049, 264, 272),
    # enough tiles for the 256-column kernels: every CTA several, ragged on both sides
    (3333, 1800, 400), (5001, 1032, 2064), (19999, 136, 272), (9800, 520, 16), (2500, 2568, 1168),
]


@pytest.mark.parametrize("mode", ["auto", "promote", "native"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(bs, M, N, K, mode):
    p = Product(M, N, K, seed=M * 31 + N + K, pow2=mode == "native")
    whole, C = _guarded(M, N)
    bs.fp8_gemm_block128(*p.on(DEV), C, mode={"auto": None, "promote": bs.FP8_PATH_PROMOTE,
                                              "native": bs.FP8_PATH_NATIVE}[mode])
    torch.cuda.synchronize()
    assert bs.fp8_status_query() == 0
    assert torch.all(whole[0] == -7.0) and torch.all(whole[-1] == -7.0), "a row outside of C was written"
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(C), Cr, T, f"block128 {mode} {M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(3000, 1800, 272), (300, 264, 400)])
def test_native_reports_other_scales(bs, M, N, K):
    """Where the block-scaled MMA runs, a scale that is not a power of two is reported;
    other forms multiply by it."""
    p = Product(M, N, K, seed=3, pow2=True)
    p.sA[M // 2, 0] = 3.0
    C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(*p.on(DEV), C, mode=bs.FP8_PATH_NATIVE)
    torch.cuda.synchronize()
    status = bs.fp8_status_query()
    assert status == (bs._abi.FP8_ERR_SCALE if M == 3000 else 0)
    keep = np.arange(M) != M // 2 if status else np.ones(M, bool)
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(C)[keep], Cr[keep], T[keep], f"native other scales {M}")


def test_native_equals_promotion_on_exact_sums(bs):
    """Codes and scales whose sums fp32 holds exactly: every path gives the same bits."""
    M, N, K = 3000, 1800, 528
    g = torch.Generator().manual_seed(6)
    one = torch.tensor([0x00, 0x38, 0xB8], dtype=torch.uint8)   # 0, 1, -1
    A = one[torch.randint(0, 3, (M, K), generator=g)].to(DEV)
    B = one[torch.randint(0, 3, (N, K), generator=g)].to(DEV)
    sA = torch.exp2(torch.randint(-2, 3, (M, 5), generator=g).float()).to(DEV)
    sB = torch.exp2(torch.randint(-2, 3, (15, 5), generator=g).float()).to(DEV)
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    for C, mode in zip(outs, (None, bs.FP8_PATH_NATIVE, bs.FP8_PATH_PROMOTE)):
        bs.fp8_gemm_block128(A, sA, B, sB, C, mode=mode)
    torch.cuda.synchronize()
    assert bs.fp8_status_query() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("mode", ["auto", "native", "split"])
def test_withheld_stage_runs_out(bs, mode):
    """A load that never comes: the bounded wait is reported, the next call is right."""
    M, N, K = (100, 264, 4112) if mode == "split" else (3000, 1800, 1040)
    p = Product(M, N, K, seed=4, pow2=True)
    ops = p.on(DEV)
    m = bs.FP8_PATH_NATIVE if mode == "native" else None
    C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(*ops, C, mode=m)
    torch.cuda.synchronize()
    try:
        bs.fp8_debug_set(bs.FP8_DEBUG_WAIT_LIMIT_CYCLES, 20_000_000)
        bs.fp8_debug_set(bs.FP8_DEBUG_WITHHOLD_STAGE, 5)
        bs.fp8_gemm_block128(*ops, C, mode=m)
        torch.cuda.synchronize()
        assert bs.fp8_status_query() == bs._abi.FP8_ERR_TIMEOUT
    finally:
        bs.fp8_debug_set(bs.FP8_DEBUG_WITHHOLD_STAGE, -1)
        bs.fp8_debug_set(bs.FP8_DEBUG_WAIT_LIMIT_CYCLES, 0)
    bs.fp8_gemm_block128(*ops, C, mode=m)
    torch.cuda.synchronize()
    assert bs.fp8_status_query() == 0
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(C), Cr, T, f"block128 after a timeout {mode}")


def test_zero_inner_size(bs):
    C = torch.full((5, 24), 3.0, dtype=torch.bfloat16, device=DEV)
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)   # noqa: E731
    f = lambda *s: torch.zeros(*s, device=DEV)                      # noqa: E731
    bs.fp8_gemm_block128(z(5, 0), f(5, 0), z(24, 0), f(1, 0), C)
    torch.cuda.synchronize()
    assert torch.all(C == 0)


@pytest.mark.parametrize("mode", ["auto", "promote", "native"])
@pytest.mark.parametrize("M,N,K", [(5, 264, 400), (130, 264, 656), (1100, 1032, 528)])
def test_extreme_scales(bs, M, N, K, mode):
    """Zero, tiny and large scales, all-zero rows, the largest codes."""
    p = Product(M, N, K, seed=5, pow2=mode == "native")
    p.A[0] = 0x7E
    p.B[3] = 0xFE
    p.A[M - 1] = 0
    p.sA[0] = 2.0 ** -40
    p.sA[1 % M] = 2.0 ** 30
    if mode != "native":
        p.sA[2] = 0.0
        p.sB[-1, 0] = 0.0
    C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(*p.on(DEV), C, mode={"auto": None, "promote": bs.FP8_PATH_PROMOTE,
                                              "native": bs.FP8_PATH_NATIVE}[mode])
    torch.cuda.synchronize()
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(C), Cr, T, f"block128 extreme {mode} {M}")


def test_rows_do_not_depend_on_the_batch_when_pinned(bs):
    p = Product(300, 264, 1168, seed=11)
    A, sA, B, sB = p.on(DEV)
    full = torch.empty(300, 264, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(A, sA, B, sB, full, mode=bs.FP8_PATH_PROMOTE)
    for m in (1, 7, 64, 129):
        C = torch.empty(m, 264, dtype=torch.bfloat16, device=DEV)
        bs.fp8_gemm_block128(A[:m], sA[:m], B, sB, C, mode=bs.FP8_PATH_PROMOTE)
        torch.cuda.synchronize()
        assert torch.equal(C.view(torch.int16), full[:m].view(torch.int16)), m


def test_rows_do_not_depend_on_the_tile_width_when_pinned(bs):
    """Enough rows for the 256-column tiles against few rows (128 columns)."""
    M, N, K = 6000, 1032, 1168
    p = Product(M, N, K, seed=15)
    A, sA, B, sB = p.on(DEV)
    full = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(A, sA, B, sB, full, mode=bs.FP8_PATH_PROMOTE)
    for a, m in ((0, 100), (3000, 1), (5800, 200)):
        C = torch.empty(m, N, dtype=torch.bfloat16, device=DEV)
        bs.fp8_gemm_block128(A[a:a + m], sA[a:a + m], B, sB, C, mode=bs.FP8_PATH_PROMOTE)
        torch.cuda.synchronize()
        assert torch.equal(C.view(torch.int16), full[a:a + m].view(torch.int16)), (a, m)


@pytest.mark.parametrize("M", [1, 20, 100, 600])
def test_a_call_repeats_bit_for_bit(bs, M):
    p = Product(M, 520, 2064, seed=12)
    ops = p.on(DEV)
    outs = [torch.empty(M, 520, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    for C in outs:
        bs.fp8_gemm_block128(*ops, C)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0].view(torch.int16), C.view(torch.int16)) for C in outs[1:])


def test_other_stream(bs):
    """The operands are made on a side stream and used there."""
    p = Product(70, 264, 528, seed=13)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        ops = p.on(DEV)
        C = torch.empty(70, 264, dtype=torch.bfloat16, device=DEV)
        bs.fp8_gemm_block128(*ops, C)
    side.synchronize()
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(C), Cr, T, "block128 side stream")


def _experts(bs, counts, N, K, mode=None, seed=1, lead=0, tail=0, pow2=False):
    """`lead` and `tail` rows belong to no expert and stay untouched."""
    E, T = len(counts), sum(counts) + lead + tail
    p = Product(T, N, K, seed=seed, E=E, pow2=pow2)
    off = [lead] + [lead + c for c in itertools.accumulate(counts)]
    C = torch.full((T, N), -7.0, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_experts(*p.on(DEV), C, torch.tensor(off, dtype=torch.int32, device=DEV), mode=mode)
    torch.cuda.synchronize()
    assert bs.fp8_status_query() == 0
    assert torch.all(C[:lead] == -7.0) and torch.all(C[off[-1]:] == -7.0), "a row of no expert was written"
    got = bf16_to_f64(C)
    for e, c in enumerate(counts):
        if c:
            r = slice(off[e], off[e + 1])
            Cr, Tm = product(p.A[r], p.sA[r], p.B[e], p.sB[e])
            check(got[r], Cr, Tm, f"experts {E}x{N}x{K} {mode} e{e}")
    return p, off, C


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 16), ([0, 3, 0, 1, 0, 0, 9], 136, 272), ([5, 0, 64, 33], 264, 528), ([0, 0, 130, 1, 0, 257], 392, 400),
    ([128] * 4, 256, 512), ([300, 1, 0, 511, 129], 520, 656), ([1] * 40, 128, 144), ([0] * 9 + [2], 24, 128),
    ([2, 0, 900, 0, 0, 140], 1032, 272),
    ([700, 0, 1, 2000, 129, 64, 33, 1500], 1288, 528), ([1] * 30 + [40] * 30, 1032, 272), ([9000, 11000], 264, 656),
])
def test_experts(bs, counts, N, K, mode):
    _experts(bs, counts, N, K, mode=mode, pow2=mode == 1)


def test_experts_rows_outside_the_table(bs):
    _experts(bs, [3, 0, 140], 264, 272, lead=5, tail=9)
    _experts(bs, [3, 0, 2, 1], 264, 272, lead=2, tail=3)


def test_experts_none_has_rows(bs):
    _experts(bs, [0, 0, 0], 128, 128, lead=4)


def test_many_experts(bs):
    rng = np.random.default_rng(3)
    _experts(bs, [int(v) for v in rng.integers(0, 3, 700)], 16, 32, seed=3)
    _experts(bs, [0] * 1000 + [40] + [0] * 23, 16, 32, seed=4)


def test_experts_equal_the_single_product_when_pinned(bs):
    p, off, C = _experts(bs, [70, 0, 129, 3], 264, 528, mode=2)
    A, sA, B, sB = p.on(DEV)
    for e in range(4):
        r = slice(off[e], off[e + 1])
        one = torch.empty(off[e + 1] - off[e], 264, dtype=torch.bfloat16, device=DEV)
        bs.fp8_gemm_block128(A[r], sA[r], B[e], sB[e], one, mode=bs.FP8_PATH_PROMOTE)
        torch.cuda.synchronize()
        assert torch.equal(one.view(torch.int16), C[r].view(torch.int16)), e


@pytest.mark.parametrize("T", [6, 300])
def test_experts_bad_table_is_clamped_and_reported(bs, T):
    p = Product(T, 136, 272, seed=8, E=3)
    for off in ([0, T + 40, T + 50, T + 60], [-5, 2, 4, T], [0, 4, 2, 2]):
        C = torch.full((T, 136), -7.0, dtype=torch.bfloat16, device=DEV)
        bs.fp8_gemm_experts(*p.on(DEV), C, torch.tensor(off, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        assert bs.fp8_status_query() == bs._abi.FP8_ERR_RECORD, off
        assert bs.fp8_status_query() == 0


def test_experts_overlapping_table_ends(bs):
    """Every expert claims all rows: clamped to disjoint ranges (tiles and split tiles),
    reported, nothing written outside of C."""
    for T, N, mode in ((900, 264, None), (40, 136, None), (3000, 1032, 1)):
        E = 6
        p = Product(T, N, 272, seed=10, E=E, pow2=True)
        whole, C = _guarded(T, N)
        bs.fp8_gemm_experts(*p.on(DEV), C, torch.tensor([0, T, 0, T, 0, T, 0], dtype=torch.int32, device=DEV), mode=mode)
        torch.cuda.synchronize()
        assert bs.fp8_status_query() == bs._abi.FP8_ERR_RECORD
        assert torch.all(whole[0] == -7.0) and torch.all(whole[-1] == -7.0)
        Cr, Tm = product(p.A, p.sA, p.B[0], p.sB[0])
        check(bf16_to_f64(C), Cr, Tm, f"experts overlapping {T}")


def test_experts_graph_follows_the_table(bs):
    """One capture; the routing changes between replays."""
    N, K, T, E = 264, 272, 200, 4
    p = Product(T, N, K, seed=9, E=E)
    ops = p.on(DEV)
    C = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 50, 50, 150, 200], dtype=torch.int32, device=DEV)
    bs.fp8_gemm_experts(*ops, C, off)   # set-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.fp8_gemm_experts(*ops, C, off)
    for table in ([0, 50, 50, 150, 200], [0, 0, 199, 199, 200], [0, 1, 2, 3, 200]):
        off.copy_(torch.tensor(table, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = bf16_to_f64(C)
        for e, (a, b) in enumerate(zip(table, table[1:])):
            if b > a:
                Cr, Tm = product(p.A[a:b], p.sA[a:b], p.B[e], p.sB[e])
                check(got[a:b], Cr, Tm, f"experts graph {table} e{e}")
    del graph


@pytest.mark.parametrize("mode", ["auto", "native"])
def test_offsets_past_32_bits(bs, mode):
    """Operands and outputs whose byte and element offsets pass 2^31: experts with
    70000 rows in all, and 33 experts of 70 MB; sampled rows."""
    N, K, E = 32768, 64, 2
    T = 70000
    g = torch.Generator(device=DEV).manual_seed(2)
    pow2 = mode == "native"
    A = torch.randn(T, K, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    B = torch.randn(E * N, K, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8).view(E, N, K)
    sA = torch.rand(T, 1, generator=g, device=DEV) + 0.5
    sB = torch.rand(E, N // 128, 1, generator=g, device=DEV) + 0.5
    if pow2:
        sA, sB = torch.exp2(torch.floor(sA * 4)), torch.exp2(torch.floor(sB * 4))
    C = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    off = [0, 66000, T]
    bs.fp8_gemm_experts(A, sA, B, sB, C, torch.tensor(off, dtype=torch.int32, device=DEV),
                        mode=bs.FP8_PATH_NATIVE if pow2 else None)
    torch.cuda.synchronize()
    for r in (0, 32767, 32768, 65535, 65536, 65999, 66000, 69999):
        e = int(r >= 66000)
        Cr, Tm = product(A[r:r + 1].cpu(), sA[r:r + 1].cpu(), B[e].cpu(), sB[e].cpu())
        check(bf16_to_f64(C[r:r + 1]), Cr, Tm, f"experts past 2^31 {mode} row {r}")


def test_weights_past_32_bits(bs):
    E, N, K = 80, 4096, 7168
    g = torch.Generator(device=DEV).manual_seed(4)
    B = torch.randint(0, 126, (E, N, K), generator=g, device=DEV, dtype=torch.uint8)
    sB = torch.rand(E, N // 128, K // 128, generator=g, device=DEV) + 0.5
    counts = [0] * E
    counts[0], counts[75], counts[79] = 3, 40, 1
    T = sum(counts)
    A = torch.randn(T, K, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    sA = torch.rand(T, K // 128, generator=g, device=DEV)
    off = [0] + list(itertools.accumulate(counts))
    C = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_experts(A, sA, B, sB, C, torch.tensor(off, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for e in (0, 75, 79):
        r = slice(off[e], off[e + 1])
        Cr, Tm = product(A[r].cpu(), sA[r].cpu(), B[e].cpu(), sB[e].cpu())
        check(bf16_to_f64(C[r]), Cr, Tm, f"experts weights past 2^31 e{e}")
