"""The 128-granular product with bias, activation and residual, against 64 bits, in every
form (rows, split and whole tiles, the block-scaled path)."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from tests import _block128 as ref
from tests import _fused

pytestmark = pytest.mark.gpu
ACT = dict(none=bs.FP8_ACT_NONE, relu=bs.FP8_ACT_RELU, gelu=bs.FP8_ACT_GELU, gelu_tanh=bs.FP8_ACT_GELU_TANH,
           silu=bs.FP8_ACT_SILU)


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_sm_gb300 import build
    build.build()


def operands(M, N, K, seed, pow2=False):
    p = ref.Product(M, N, K, seed, pow2)
    # sums of a few units, so that the activations are met where they bend
    p.sB = p.sB / 8 if pow2 else p.sB / (2 * K ** 0.5)
    g = torch.Generator().manual_seed(seed + 1)
    return p.on("cuda"), torch.randn(N, generator=g).cuda(), torch.randn(M, N, generator=g).to(torch.bfloat16).cuda()


def compare(out, C, bound, what):
    err = (out.double() - C).abs()
    assert bool((err <= bound).all()), f"{what}: worst {float((err / bound).max()):.3f} of the bound"


# M, N, K, mode: rows in one wave and many, rows in groups of 16, tiles with K split and
# not (pinned), 256-column tiles with ends inside, more than one tile for a CTA
FORMS = [(1, 4096, 512, None), (5, 4904, 144, None), (16, 520, 1040, None), (37, 8200, 272, None),
         (37, 4104, 7184, None), (150, 392, 2064, bs.FP8_PATH_PROMOTE), (1300, 3608, 272, None),
         (2500, 4360, 144, None)]


@pytest.mark.parametrize("act", _fused.ACTS)
@pytest.mark.parametrize("M,N,K,mode", FORMS)
def test_forms(M, N, K, mode, act):
    ops, bias, R = operands(M, N, K, M + N)
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT[act], residual=R, mode=mode)
    compare(C, *_fused.fused(*ops, bias, act, R), f"{M}x{N}x{K} {act}")
    assert bs.fp8_status_query() == 0


@pytest.mark.parametrize("act", _fused.ACTS)
@pytest.mark.parametrize("M,N,K", [(1300, 3608, 272), (2500, 4360, 1040), (3, 264, 256)])
def test_native(M, N, K, act):
    ops, bias, R = operands(M, N, K, M + K, pow2=True)
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bs.fp8_gemm_block128_fused(*ops, C, bias=bias.to(torch.bfloat16), act=ACT[act], residual=R,
                               mode=bs.FP8_PATH_NATIVE)
    compare(C, *_fused.fused(*ops, bias.to(torch.bfloat16), act, R), f"native {M}x{N}x{K} {act}")
    assert bs.fp8_status_query() == 0


@pytest.mark.parametrize("bias", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N,K", [(2, 136, 144), (33, 136, 400), (300, 136, 272), (1300, 3608, 144)])
def test_parts(M, N, K, bias, residual):
    ops, b, R = operands(M, N, K, M * 3 + N)
    b = None if bias is None else b.to(bias)
    R = R if residual else None
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    bs.fp8_gemm_block128_fused(*ops, C, bias=b, act=ACT["silu"], residual=R)
    compare(C, *_fused.fused(*ops, b, "silu", R), f"{M}x{N}x{K} bias {bias}")


@pytest.mark.parametrize("M,N,K,mode", FORMS + [(1300, 3608, 272, bs.FP8_PATH_NATIVE)])
def test_empty_epilogue_has_the_products_bits(M, N, K, mode):
    ops, _, _ = operands(M, N, K, 5, pow2=mode == bs.FP8_PATH_NATIVE)
    C, D = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bs.fp8_gemm_block128_fused(*ops, C, mode=mode)
    bs.fp8_gemm_block128(*ops, D, mode=mode)
    assert torch.equal(C.view(torch.int16), D.view(torch.int16))


@pytest.mark.parametrize("M,N,K", [(1, 264, 144), (40, 264, 2064), (1300, 3608, 144)])
def test_residual_in_place(M, N, K):
    ops, bias, R = operands(M, N, K, 11)
    want, bound = _fused.fused(*ops, bias, "gelu", R)
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT["gelu"], residual=R)
    bs.fp8_gemm_block128_fused(*ops, R, bias=bias, act=ACT["gelu"], residual=R)
    assert torch.equal(C.view(torch.int16), R.view(torch.int16))
    compare(R, want, bound, "in place")


@pytest.mark.parametrize("M", [1, 9, 700])
def test_no_k(M):
    A, sA = torch.empty(M, 0, dtype=torch.uint8, device="cuda"), torch.empty(M, 0, device="cuda")
    B, sB = torch.empty(264, 0, dtype=torch.uint8, device="cuda"), torch.empty(3, 0, device="cuda")
    g = torch.Generator().manual_seed(M)
    bias, R = torch.randn(264, generator=g).cuda(), torch.randn(M, 264, generator=g).to(torch.bfloat16).cuda()
    C = torch.empty(M, 264, dtype=torch.bfloat16, device="cuda")
    bs.fp8_gemm_block128_fused(A, sA, B, sB, C, bias=bias, act=ACT["gelu"], residual=R)
    compare(C, *_fused.fused(A, sA, B, sB, bias, "gelu", R), "no K")


@pytest.mark.parametrize("act", _fused.ACTS)
def test_activation_over_its_range(act):
    """The whole range of bf16 (no K: the bias alone goes through the activation)."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    y = bits[bits.float().isfinite()]
    y = torch.cat([y, y.new_zeros(-y.numel() % 8)]).cuda()
    N = y.numel()
    z = torch.empty(1, 0, device="cuda")
    C = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    bs.fp8_gemm_block128_fused(z.to(torch.uint8), z, torch.empty(N, 0, dtype=torch.uint8, device="cuda"),
                               torch.empty(-(-N // 128), 0, device="cuda"), C, bias=y, act=ACT[act])
    f = _fused.activation(y.double(), act)
    f = torch.where(f.isnan(), torch.zeros_like(f), f)   # y^3 past the doubles' range: the tail is 0
    # 2^-8 for the rounding, 2^-14 for the activation; below 2^-126 the steps are subnormal,
    # and there the fp32 factors lose up to |y| 2^-126 more (y < 2^4 times 2^-149, doubled)
    bound = (2.0 ** -8 + 2.0 ** -14) * f.abs() + 2.0 ** -133
    compare(C[0], f, bound, act)


@pytest.mark.parametrize("M,N,K,mode", [(1, 264, 144, None), (40, 264, 2064, None), (300, 136, 272, None),
                                        (1300, 3608, 144, None), (1300, 3608, 144, bs.FP8_PATH_NATIVE)])
def test_nan_and_infinity_stay_in_their_place(M, N, K, mode):
    ops, bias, R = operands(M, N, K, 17, pow2=True)
    C, D = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT["relu"], residual=R, mode=mode)
    bias[7], R[M - 1, 9], R[0, 12] = float("nan"), float("-inf"), float("nan")
    bs.fp8_gemm_block128_fused(*ops, D, bias=bias, act=ACT["relu"], residual=R, mode=mode)
    same = torch.ones(M, N, dtype=torch.bool, device="cuda")
    same[:, 7], same[M - 1, 9], same[0, 12] = False, False, False
    assert torch.equal(C[same], D[same])
    assert bool(D[:, 7].isnan().all()) and float(D[M - 1, 9]) == float("-inf") and bool(D[0, 12].isnan())


def test_replayed_in_a_graph_and_on_another_stream():
    M, N, K = 24, 520, 1040
    ops, bias, R = operands(M, N, K, 23)
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT["silu"], residual=R)
    first = C.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT["silu"], residual=R)
    C.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, first)
    R.copy_(torch.randn(M, N, device="cuda"))
    graph.replay()
    D = torch.empty_like(C)
    side.wait_stream(torch.cuda.current_stream())
    bs.fp8_gemm_block128_fused(*ops, D, bias=bias, act=ACT["silu"], residual=R, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(C, D)
    del graph


@pytest.mark.parametrize("bias,residual", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K,mode", [(2500, 4360, 144, None), (2500, 4360, 144, bs.FP8_PATH_NATIVE),
                                        (150, 19464, 272, bs.FP8_PATH_PROMOTE)])
def test_many_tiles_of_a_cta_in_place(M, N, K, mode, bias, residual):
    """More tiles than CTAs: what is staged for one tile is not taken for another's."""
    ops, b, R = operands(M, N, K, 29, pow2=mode == bs.FP8_PATH_NATIVE)
    b = b if bias else None
    want, bound = _fused.fused(*ops, b, "none", R if residual else None)
    bs.fp8_gemm_block128_fused(*ops, R, bias=b, residual=R if residual else None, mode=mode)
    compare(R, want, bound, f"{M}x{N}x{K}")


@pytest.mark.parametrize("stage", [0, 2, 7])
def test_withheld_stage_times_out_cleanly(stage):
    """Waits that run out are reported, the kernel returns, and the next call is right."""
    M, N, K = 1300, 3608, 1040
    ops, bias, R = operands(M, N, K, 31)
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert bs.fp8_status_query() == 0
    bs.fp8_debug_set(bs.FP8_DEBUG_WAIT_LIMIT_CYCLES, 20_000_000)   # ~10 ms
    bs.fp8_debug_set(bs.FP8_DEBUG_WITHHOLD_STAGE, stage)
    try:
        bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT["silu"], residual=R)
        torch.cuda.synchronize()
        assert bs.fp8_status_query() == bs._abi.FP8_ERR_TIMEOUT
    finally:
        bs.fp8_debug_set(bs.FP8_DEBUG_WITHHOLD_STAGE, -1)
        bs.fp8_debug_set(bs.FP8_DEBUG_WAIT_LIMIT_CYCLES, 0)
    bs.fp8_gemm_block128_fused(*ops, C, bias=bias, act=ACT["silu"], residual=R)
    compare(C, *_fused.fused(*ops, bias, "silu", R), "after the time-out")
    assert bs.fp8_status_query() == 0
