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
def test_infinite_residual(M, N, K, mode, act):
    ops, bias, R = operands(M, N, K)
    clean = call(ops, bias, act, R, mode)
    R[0, 8], R[M - 1, 17] = INF, -INF
    got = call(ops, bias, act, R, mode)
    assert float(got[0, 8]) == INF and float(got[M - 1, 17]) == -INF
    got[0, 8], got[M - 1, 17] = clean[0, 8], clean[M - 1, 17]
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))
