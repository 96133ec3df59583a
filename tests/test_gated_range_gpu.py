"""The gated quantizer over the whole range of bf16 gates and ups, against silu(gate) up in
64 bits.

Error of the kernel's y, at most: the sigmoid's exponential, which for gates of -64 and
below is the square of one taken at half the argument (2 ulp of 2^-23, twice: 2^-21; its
correction and the square, three roundings of 2^-24), 1 + e and the reciprocal (2^-24 and
2^-23), the products (four of 2^-24): together
2^-21 + 2^-23 + 8 * 2^-24 = 1.125 * 2^-20.  The quotient by the scale adds an ulp, 2^-23:
1.25 * 2^-20.  A code may be half a step and that much of the value off; a scale that much of
itself, or, rounded up to a power of two, one power where the unrounded one is that near."""
import numpy as np
import pytest
import torch

from tests._block128 import TABLE, blocks, quantized

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 1.25 * 2.0 ** -20
MAX = float(torch.finfo(torch.bfloat16).max)


@pytest.fixture(scope="module")
def bs():
    import block_scaled_fp8_sm_gb300 as mod
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    mod.library()
    return mod


def _silu_mul(gate, up):
    g, u = gate.double().numpy(), up.double().numpy()
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def _check(q, s, y, pow2, what):
    """Pieces of finite y; one below 2^-100 counts as all zero by definition."""
    y = y.copy()
    for b in range(blocks(y.shape[1])):
        piece = y[:, b * 128:(b + 1) * 128]
        piece[np.abs(piece).max(axis=1) < 2.0 ** -100] = 0.0
    got, got_s = TABLE[q.cpu().numpy()], s.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), f"{what}: NaN codes"
    _, ws = quantized(y, False)
    if pow2:
        near = [quantized(y * (1 + d), True)[1] for d in (-TOL, 0.0, TOL)]
        assert np.all((got_s == near[0]) | (got_s == near[1]) | (got_s == near[2])), what
    else:
        assert np.all(np.abs(got_s - ws) <= TOL * ws), what
    v = y / np.repeat(got_s, 128, 1)[:, :y.shape[1]]
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    off = np.abs(got - np.clip(v, -448, 448)) - (step / 2 + TOL * np.abs(v))
    assert np.all(off <= 0), f"{what}: {int((off > 0).sum())} codes, first at {np.argwhere(off > 0)[0]}"


def _run(bs, gate, up, pow2, what):
    x = torch.cat([gate, up], dim=1).to(torch.bfloat16)
    K = gate.shape[1]
    q, s = bs.fp8_swiglu_quantize_tokens(x.to(DEV), pow2=pow2)
    torch.cuda.synchronize()
    _check(q, s, _silu_mul(x[:, :K], x[:, K:]), pow2, what)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("up", [1.0, 1e-3, -1e-30, 0.0])
def test_largest_gates(bs, up, pow2):
    """|gate| log2(e) passes the largest fp32 number from 2.36e38 on."""
    big = torch.tensor([2.3e38, 2.4e38, 3e38, MAX, -2.3e38, -2.4e38, -3e38, -MAX])
    g = torch.Generator().manual_seed(1)
    gate = torch.randn(9, 272, generator=g)
    gate[:8, 5], gate[:8, 140] = big, big.flip(0)
    gate[8] = -MAX                        # nothing but zeros
    u = torch.randn(9, 272, generator=g).sign() * up
    _run(bs, gate, u, pow2, f"largest gates, up {up}")


@pytest.mark.parametrize("pow2", [False, True])
def test_small_sigmoids_keep_their_precision(bs, pow2):
    """Gates below -87, whose exponential fp32 cannot hold in full, with ups that bring the
    result back into range; every piece has values of one magnitude."""
    g = torch.Generator().manual_seed(2)
    base = torch.linspace(-172, -84, 64)[:, None]
    gate = base + torch.randn(64, 384, generator=g) * 0.3
    up = torch.randn(64, 384, generator=g).clamp(-3, 3) * torch.logspace(24, 38, 64).flip(0)[:, None]
    _run(bs, gate, up, pow2, "small sigmoids")


@pytest.mark.parametrize("pow2", [False, True])
def test_factors_at_the_ends_of_the_range(bs, pow2):
    """Subnormal gates with large ups and the other way round, and products next to the
    largest fp32 number."""
    g = torch.Generator().manual_seed(3)
    n = lambda: torch.randn(4, 256, generator=g)   # noqa: E731
    small, large = torch.tensor([2.0 ** -133, 2.0 ** -130, 2.0 ** -127, 2.0 ** -126])[:, None], 1e30
    _run(bs, n() * small, n() * large, pow2, "subnormal gates")
    _run(bs, n().abs() * large, n() * small, pow2, "subnormal ups")
    _run(bs, 0.5 + n().abs() / 8, n().sign() * MAX, pow2, "largest ups")   # silu(1.4) < 1


@pytest.mark.parametrize("pow2", [False, True])
def test_products_past_the_largest_number(bs, pow2):
    """Finite gates and ups whose product fp32 cannot hold: as the quotient by an infinite
    scale gives, NaN for these values and zero for the rest of their piece."""
    g = torch.Generator().manual_seed(4)
    gate, up = torch.randn(6, 400, generator=g), torch.randn(6, 400, generator=g)
    gate[1, 130], up[1, 130] = 1e30, -1e30
    gate[4, 399], up[4, 399] = 3.0, MAX
    x = torch.cat([gate, up], dim=1).to(torch.bfloat16)
    q, s = bs.fp8_swiglu_quantize_tokens(x.to(DEV), pow2=pow2)
    torch.cuda.synchronize()
    got, got_s = TABLE[q.cpu().numpy()], s.cpu().numpy()
    want = np.zeros((6, 400))
    want[1, 130] = want[4, 399] = np.nan
    for row, piece in ((1, slice(128, 256)), (4, slice(384, 400))):
        assert got_s[row, piece.start // 128] == np.inf
        assert np.array_equal(got[row, piece], want[row, piece], equal_nan=True), (row, got[row, piece])
    assert int(np.isinf(got_s).sum()) == 2
    y = _silu_mul(x[:, :400], x[:, 400:])
    for b in range(4):
        keep = ~np.isinf(got_s[:, b])
        cols = slice(b * 128, min(400, b * 128 + 128))
        _check(q[keep][:, cols], s[keep][:, b:b + 1], y[keep, cols], pow2, f"beside infinite values, piece {b}")


@pytest.mark.parametrize("low,high", [(-60, -1), (-8, 8), (0, 20)])
def test_ordinary_gates_are_as_exact_as_plain_arithmetic(bs, low, high):
    """One value to a piece, read off its scale: the rms error against 64 bits, next to that
    of the formula in plain fp32 operations.  Those round four times beside their exponential
    (sum, quotient, product, scale); the kernel eight times at most (the exponential's
    correction, the sum, a reciprocal of one ulp for two, three products, the scale): at most
    sqrt(8 / 4) times the error, 1.42; 1.5 is accepted."""
    g = torch.Generator().manual_seed(5)
    P = 1 << 17
    gate = (torch.rand(P, generator=g) * (high - low) + low).to(torch.bfloat16)
    up = torch.randn(P, generator=g).to(torch.bfloat16)
    x = torch.zeros(P // 16, 2, 16, 128, dtype=torch.bfloat16)
    x[:, 0, :, 5], x[:, 1, :, 5] = gate.view(-1, 16), up.view(-1, 16)
    _, s = bs.fp8_swiglu_quantize_tokens(x.view(P // 16, -1).to(DEV))
    y = np.abs(_silu_mul(gate, up)) / 448.0
    gate, up = gate.to(DEV).float(), up.to(DEV).float()
    plain = (gate / (1 + torch.exp(-gate)) * up).abs()
    plain = (plain / torch.full_like(plain, 448.0)).cpu().numpy().astype(np.float64)
    keep = y > 2.0 ** -90
    assert keep.mean() > 0.9
    own, plain = (float(np.sqrt(np.mean(((v - y) / np.where(keep, y, 1.0))[keep] ** 2)))
                  for v in (s.cpu().numpy().astype(np.float64).ravel(), plain))
    assert own <= 1.5 * plain, (own, plain)
