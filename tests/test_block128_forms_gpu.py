"""Every form of the 128-granular products that the dispatch rules can pick, the streams they
run on, and the quantizer's option pairs, against 64 bits."""
import itertools

import numpy as np
import pytest
import torch

from tests._accept import bf16_to_f64, check
from tests._block128 import Product, product, quantized
from tests.test_gated_range_gpu import _run as gated_run
from tests.test_quant_tokens_gpu import SIZES, _exact, _x

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SMS = 152


@pytest.fixture(scope="module")
def bs():
    import block_scaled_fp8_sm_gb300 as mod
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    mod.library()
    return mod


def _strips(N):
    return -(-N // 16)


# few rows and so many columns that the CTAs do not fit two (eight warps) to an SM: the
# four-warp forms, with all CTAs on the GPU at once and with more; N ends inside a strip
WIDE = [(1, 5000, 272), (8, 9720, 400), (7, 16392, 272), (8, 16384, 1040),
        (16, 8200, 272), (9, 9720, 144), (13, 20008, 272), (33, 2568, 144), (64, 2568, 144), (64, 4104, 144)]


@pytest.mark.parametrize("mode", [None, 1])
@pytest.mark.parametrize("M,N,K", WIDE)
def test_few_rows_many_columns(bs, M, N, K, mode):
    groups = 1 if M <= 8 else -(-M // 16)
    assert _strips(N) * groups > 2 * SMS and N * K * (24 * groups - 14) <= 330_000_000
    p = Product(M, N, K, seed=M + N, pow2=mode == 1)
    whole = torch.full((M + 2, N), -7.0, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(*p.on(DEV), whole[1:M + 1], mode=mode)
    torch.cuda.synchronize()
    assert bs.fp8_status_query() == 0
    assert bool((whole[0] == -7.0).all() and (whole[-1] == -7.0).all())
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(whole[1:M + 1]), Cr, T, f"few rows, many columns {mode} {M}x{N}x{K}")


def test_both_kinds_of_launch_are_covered():
    on_gpu = [_strips(n) * (1 if m <= 8 else -(-m // 16)) <= 4 * SMS for m, n, _ in WIDE]
    assert {(m > 8, fits) for (m, _, _), fits in zip(WIDE, on_gpu)} == set(itertools.product((False, True), repeat=2))


@pytest.mark.parametrize("mode", ["auto", "promote", "native"])
@pytest.mark.parametrize("M,N,K", [(3000, 1800, 528), (9800, 520, 272)])
def test_extreme_scales_in_wide_tiles(bs, M, N, K, mode):
    """Tiny and large scales, all-zero rows and the largest codes where 256-column tiles, or
    the block-scaled MMA, run; zero scales where any scale is allowed."""
    assert -(-M // 128) * -(-N // 256) >= SMS
    p = Product(M, N, K, seed=5, pow2=mode == "native")
    p.A[0] = 0x7E
    p.B[3] = 0xFE
    p.A[M - 1], p.A[300:700] = 0, 0
    p.sA[0] = 2.0 ** -40
    p.sA[1] = 2.0 ** 30
    p.sA[128], p.sB[1, 0] = 2.0 ** -60, 2.0 ** 20
    if mode != "native":
        p.sA[2] = 0.0
        p.sB[-1, 0] = 0.0
    C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(*p.on(DEV), C, mode={"auto": None, "promote": bs.FP8_PATH_PROMOTE,
                                              "native": bs.FP8_PATH_NATIVE}[mode])
    torch.cuda.synchronize()
    assert bs.fp8_status_query() == 0
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(C), Cr, T, f"extreme scales, wide tiles {mode} {M}")


def _on_a_side_stream(sources, call, explicit):
    """`call(operands, stream)` with operands that a copy on a side stream fills late: the
    copies come after a sleep on that stream, and are of this device (they do not wait for
    the host).  A call on any other stream would see zeros.  Its outputs, read after the
    side stream alone is done."""
    temps = [t.to(DEV) for t in sources]
    ops = [torch.zeros_like(t) for t in temps]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
        for o, t in zip(ops, temps):
            o.copy_(t, non_blocking=True)
        if not explicit:
            out = call(ops, None)
    if explicit:   # the current stream is the default one
        out = call(ops, side)
    side.synchronize()
    with torch.cuda.stream(side):
        return [o.cpu() for o in out]


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("M", [1, 70, 600])
def test_product_runs_on_the_given_stream(bs, M, explicit):
    p = Product(M, 264, 528, seed=13)
    C = torch.zeros(M, 264, dtype=torch.bfloat16, device=DEV)
    out, = _on_a_side_stream((p.A, p.sA, p.B, p.sB), lambda o, s: [bs.fp8_gemm_block128(*o, C, stream=s)], explicit)
    Cr, T = product(p.A, p.sA, p.B, p.sB)
    check(bf16_to_f64(out), Cr, T, f"block128 on a side stream {M}")


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("counts", [[2, 0, 3], [100, 0, 129]])
def test_experts_run_on_the_given_stream(bs, counts, explicit):
    T = sum(counts)
    p = Product(T, 264, 528, seed=14, E=3)
    off = [0] + list(itertools.accumulate(counts))
    C = torch.zeros(T, 264, dtype=torch.bfloat16, device=DEV)
    out, = _on_a_side_stream((p.A, p.sA, p.B, p.sB, torch.tensor(off, dtype=torch.int32)),
                             lambda o, s: [bs.fp8_gemm_experts(*o[:4], C, o[4], stream=s)], explicit)
    for e in (0, 2):
        r = slice(off[e], off[e + 1])
        Cr, Tm = product(p.A[r], p.sA[r], p.B[e], p.sB[e])
        check(bf16_to_f64(out)[r], Cr, Tm, f"experts on a side stream {T} e{e}")


@pytest.mark.parametrize("explicit", [False, True])
def test_quantizers_run_on_the_given_stream(bs, explicit):
    x = _x(300, 528, 2)
    q, s = _on_a_side_stream((x,), lambda o, st: bs.fp8_quantize_tokens(o[0], stream=st), explicit)
    _exact(q, s, quantized(x.double().numpy()), "side stream")
    h = torch.randn(300, 1056, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    q, s = _on_a_side_stream((h,), lambda o, st: bs.fp8_swiglu_quantize_tokens(o[0], stream=st), explicit)
    want = bs.fp8_swiglu_quantize_tokens(h.to(DEV))
    assert torch.equal(q, want[0].cpu()) and torch.equal(s, want[1].cpu()) and bool((q != 0).any())


@pytest.mark.parametrize("M,K", [(1, 16), (37, 400), (1000, 2064)])
def test_gathered_with_power_of_two_scales(bs, M, K):
    x = _x(M, K, M)
    rows = torch.randint(-1, M + 1, (3 * M + 2,), generator=torch.Generator().manual_seed(M), dtype=torch.int32)
    q, s = bs.fp8_quantize_tokens(x.to(DEV), rows=rows.to(DEV), pow2=True)
    torch.cuda.synchronize()
    y = np.stack([x[r].double().numpy() if 0 <= r < M else np.zeros(K) for r in rows.tolist()])
    _exact(q, s, quantized(y, True), f"gathered, powers of two {M}x{K}")


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_gated_scales_are_exact_or_next_to_a_power(bs, M, K, pow2):
    """Every scale is checked (a power of two may differ from the reference's only where the
    unrounded scale lies next to one)."""
    g = torch.Generator().manual_seed(M * 5 + K)
    gated_run(bs, torch.randn(M, K, generator=g) * 3, torch.randn(M, K, generator=g), pow2, f"gated scales {M}x{K}")
