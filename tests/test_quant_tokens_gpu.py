"""The per-token quantizer against its definition in 64 bits.  Plain and gathered
rows: codes and scales exactly (bf16 inputs divide exactly as the definition says).
Gated rows: silu(g) u is computed in fp32, so a scale may be off by its relative
error and a code by one step where y / s lies within that error of a rounding
boundary.  That error: exp within 2 ulp, which moves 1/(1 + exp(-g)) by at most as
much, then an addition, a division, a product and the scale's division, half an
ulp each: (2 + 4/2) 2^-23 = 2^-21, taken twice for |y| and the maximum."""
import numpy as np
import pytest
import torch

from tests._block128 import TABLE, blocks, quantized

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
REL = 2.0 ** -20


@pytest.fixture(scope="module")
def bs():
    import block_scaled_fp8_sm_gb300 as mod
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    mod.library()
    return mod


def _x(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x = torch.where(torch.rand(M, K, generator=g) < 0.005, x * 50, x)
    x = x * torch.exp2(torch.randint(-30, 30, (M, 1), generator=g).float())
    x[0, :16] = 0.0
    if M > 3:
        x[1] = 0.0                       # an all-zero token
        x[2] = 3e38                      # large
        x[3] = 1e-39                     # subnormal
        x[3, ::2] = -1e-39
    return x.to(torch.bfloat16)


def _exact(q, s, want, what):
    wq, ws = want
    assert np.array_equal(s.cpu().numpy().astype(np.float64), ws), what
    assert np.array_equal(TABLE[q.cpu().numpy()], wq), what


SIZES = [(1, 16), (1, 7168), (3, 128), (5, 144), (17, 400), (64, 2064), (333, 272), (1000, 512)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_plain(bs, M, K, pow2):
    x = _x(M, K, M + K)
    q, s = bs.fp8_quantize_tokens(x.to(DEV), pow2=pow2)
    torch.cuda.synchronize()
    _exact(q, s, quantized(x.double().numpy(), pow2), f"{M}x{K}")


@pytest.mark.parametrize("pow2", [False, True])
def test_every_bf16_value(bs, pow2):
    """All finite positive and negative bf16 values, each piece in its own binade and
    pieces that span all of them."""
    v = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.cat([v, -v])
    x = torch.cat([x.reshape(-1, 128), x.reshape(128, -1).T.contiguous()]).reshape(-1, 256)
    q, s = bs.fp8_quantize_tokens(x.to(DEV), pow2=pow2)
    torch.cuda.synchronize()
    _exact(q, s, quantized(x.double().numpy(), pow2), "every value")


@pytest.mark.parametrize("K", [16, 144, 2064])
def test_gathered(bs, K):
    x = _x(37, K, K)
    rows = [0, 36, 36, -1, 5, 37, 1, 2, 2 ** 31 - 1, -2 ** 31, 3, 3, 12]
    q, s = bs.fp8_quantize_tokens(x.to(DEV), rows=torch.tensor(rows, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    y = np.stack([x[r].double().numpy() if 0 <= r < 37 else np.zeros(K) for r in rows])
    _exact(q, s, quantized(y), f"gathered {K}")


def test_strided_rows(bs):
    x = _x(50, 1040, 7)
    view = x.to(DEV)[:, 16:16 + 528]
    q, s = bs.fp8_quantize_tokens(view)
    torch.cuda.synchronize()
    _exact(q, s, quantized(x[:, 16:544].double().numpy()), "strided")


def test_strided_outputs_are_not_overrun(bs):
    q = torch.full((7, 144), 0xAA, dtype=torch.uint8, device=DEV)
    s = torch.full((7, 2), -1.0, device=DEV)
    x = _x(5, 144, 8)
    bs.fp8_quantize_tokens(x.to(DEV), q[1:6], s[1:6])
    torch.cuda.synchronize()
    assert torch.all(q[0] == 0xAA) and torch.all(q[6] == 0xAA) and torch.all(s[0] == -1) and torch.all(s[6] == -1)
    _exact(q[1:6], s[1:6], quantized(x.double().numpy()), "inner rows")


def _near(q, s, y, pow2, what):
    """Scales within REL (or, rounded up to a power of two, one step where the
    unrounded one is within REL of it); codes equal, or next to a boundary."""
    for b in range(blocks(y.shape[1])):   # by definition: a piece below 2^-100 counts as zero
        piece = y[:, b * 128:(b + 1) * 128]
        piece[np.abs(piece).max(axis=1) < 2.0 ** -100] = 0.0
    got_s, got = s.cpu().numpy().astype(np.float64), TABLE[q.cpu().numpy()]
    wq, ws = quantized(y, pow2)
    if pow2:
        assert np.mean(got_s != ws) < 1e-3
    else:
        assert np.all(np.abs(got_s - ws) <= REL * ws), what
    full = np.repeat(got_s, 128, 1)[:, :y.shape[1]]
    v = y / full
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    assert np.all(np.abs(got - np.clip(v, -448, 448)) <= step / 2 + REL * np.abs(v)), what


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_gated(bs, M, K, pow2):
    g = torch.Generator().manual_seed(M * 3 + K)
    x = (torch.randn(M, 2 * K, generator=g) * 3).to(torch.bfloat16)
    x[0, :K] = torch.linspace(-120, 120, K).to(torch.bfloat16)   # exp overflows on one side
    if M > 2:
        x[1, :K] = 0.0
        x[2, K:] = 0.0
    q, s = bs.fp8_swiglu_quantize_tokens(x.to(DEV), pow2=pow2)
    torch.cuda.synchronize()
    gate, up = x[:, :K].double().numpy(), x[:, K:].double().numpy()
    _near(q, s, gate / (1 + np.exp(-gate)) * up, pow2, f"gated {M}x{K}")


def test_gated_strided(bs):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(20, 400, generator=g).to(torch.bfloat16)
    q, s = bs.fp8_swiglu_quantize_tokens(x.to(DEV)[:, 32:32 + 288])
    torch.cuda.synchronize()
    gate, up = x[:, 32:176].double().numpy(), x[:, 176:320].double().numpy()
    _near(q, s, gate / (1 + np.exp(-gate)) * up, False, "gated strided")


def test_feeds_the_product(bs):
    from tests._accept import bf16_to_f64, check
    from tests._block128 import Product, product
    p = Product(45, 136, 272, seed=3)
    x = _x(45, 272, 5)
    x[2], x[3] = 1.0, -1.0
    A, sA = bs.fp8_quantize_tokens(x.to(DEV))
    C = torch.empty(45, 136, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_block128(A, sA, p.B.to(DEV), p.sB.to(DEV), C)
    torch.cuda.synchronize()
    Cr, T = product(A.cpu(), sA.cpu(), p.B, p.sB)
    check(bf16_to_f64(C), Cr, T, "quantized rows through the product")


def test_offsets_past_32_bits(bs):
    M, K = 300_001, 7168
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    q, s = bs.fp8_quantize_tokens(x)
    torch.cuda.synchronize()
    for r in (0, 149796, 149797, 299593, 299594, M - 1):
        _exact(q[r:r + 1], s[r:r + 1], quantized(x[r:r + 1].cpu().double().numpy()), f"row {r}")
    assert blocks(K) == s.shape[1]
