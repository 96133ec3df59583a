"""NaN and infinities in the fused 128-granular product: what they become by the formula, and
that they stay with the outputs that they belong to, for every activation and form."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from tests import _block128 as ref
from tests import _fused

pytestmark = pytest.mark.gpu
ACT = dict(none=bs.FP8_ACT_NONE, relu=bs.FP8_ACT_RELU, gelu=bs.FP8_ACT_GELU, gelu_tanh=bs.FP8_ACT_GELU_TANH,
           silu=bs.FP8_ACT_SILU)
NAN, INF = float("nan"), float("inf")

# rows in one wave, many and groups of 16; K split; whole tiles of 128 and 256 columns, more of
# them than SMs; the block-scaled form (all with power-of-two scales, so that each takes any)
FORMS = [(1, 4096, 512, None), (5, 4904, 144, None), (16, 520, 1040, None), (100, 520, 2064, None),
         (150, 392, 2064, bs.FP8_PATH_PROMOTE), (150, 19464, 272, bs.FP8_PATH_PROMOTE), (1300, 3608, 144, None),
         (2500, 4360, 144, None), (2500, 4360, 144, bs.FP8_PATH_NATIVE)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_sm_gb300 import build
    build.build()


def operands(M, N, K):
    p = ref.Product(M, N, K, M + K, True)
    p.sB = p.sB / 8
    g = torch.Generator().manual_seed(M + N)
    return p.on("cuda"), torch.randn(N, generator=g).cuda(), torch.randn(M, N, generator=g).to(torch.bfloat16).cuda()


def call(ops, bias, act, R, mode):
    C = torch.full((ops[0].shape[0], ops[2].shape[0]), 3.0, dtype=torch.bfloat16, device="cuda")
    return bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT[act], residual=R, mode=mode)


@pytest.mark.parametrize("act", _fused.ACTS)
@pytest.mark.parametrize("M,N,K,mode", FORMS)
def test_nan_stays_in_its_column(M, N, K, mode, act):
    """In the bias, in a row of B and in a row of A; even and odd columns."""
    ops, bias, R = operands(M, N, K)
    clean = call(ops, bias, act, R, mode)
    assert bool(clean.isfinite().all())
    columns, rows = [6, 33, N - 1], [M // 2]
    bias[6], bias[33] = NAN, -NAN
    ops[2][N - 1, K // 2] = 0x7F
    ops[0][rows[0], K - 1] = 0xFF
    spoilt = call(ops, bias, act, R, mode)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[:, columns], bad[rows] = True, True
    assert bool(spoilt[bad].isnan().all())
    assert torch.equal(spoilt[~bad].view(torch.int16), clean[~bad].view(torch.int16))


@pytest.mark.parametrize("act", _fused.ACTS)
@pytest.mark.parametrize("M,N,K,mode", FORMS)
def test_infinities_by_the_formula(M, N, K, mode, act):
    """+inf stays; -inf becomes 0 by relu and 0 times infinity, NaN, by the gates."""
    ops, bias, R = operands(M, N, K)
    clean = call(ops, bias, act, R, mode)
    at = torch.tensor([0, 9, 32, N - 1], device="cuda")
    y = torch.tensor([INF, -INF, -INF, INF], device="cuda")
    bias[at] = y
    got = call(ops, bias, act, R, mode)
    want = _fused.activation(y.double(), act).float()
    assert (float(want[0]), float(want[3])) == (INF, INF)
    want = torch.where(want == 0, R[:, at].float(), want.expand(M, 4))   # relu's 0 and the residual
    torch.testing.assert_close(got[:, at].float(), want, rtol=0, atol=0, equal_nan=True)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(got[:, rest].view(torch.int16), clean[:, rest].view(torch.int16))


@pytest.mark.parametrize("act", _fused.ACTS)
@pytest.mark.parametrize("M,N,K,mode", FORMS)
def test_infinite_residual(M, N, K, mode, act):
    ops, bias, R = operands(M, N, K)
    clean = call(ops, bias, act, R, mode)
    R[0, 8], R[M - 1, 17] = INF, -INF
    got = call(ops, bias, act, R, mode)
    assert float(got[0, 8]) == INF and float(got[M - 1, 17]) == -INF
    got[0, 8], got[M - 1, 17] = clean[0, 8], clean[M - 1, 17]
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))


@pytest.mark.parametrize("act", _fused.ACTS)
def test_every_bf16_without_k(act):
    """All 65536 bf16 numbers side by side, NaN among them (no K: the bias alone)."""
    y = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    N, z = y.numel(), torch.empty(9, 0, device="cuda")
    got = bs.fp8_gemm_block128_fused(z.to(torch.uint8), z, torch.empty(N, 0, dtype=torch.uint8, device="cuda"),
                                     torch.empty(N // 128, 0, device="cuda"),
                                     torch.empty(9, N, dtype=torch.bfloat16, device="cuda"), bias=y, act=ACT[act])
    want = _fused.activation(y.double(), act)
    assert torch.equal(got.isnan(), want.isnan().expand(9, N))
    assert torch.equal(got == INF, (want > 3.3961e38).expand(9, N))   # past bf16's range: infinite
