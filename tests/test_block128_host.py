"""Argument checks of the 128-granular entry points (no GPU: every refusal comes
before a device is touched)."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from block_scaled_fp8_sm_gb300 import _abi


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    return bs.library()


def test_product_refusals(lib):
    def call(mode=0, **kw):
        a = dict(A=16, sA=16, B=16, sB=16, C=16, M=64, N=64, K=64)
        a.update(kw)
        return lib.fp8_gemm_block128_ex(a["A"], a["sA"], a["B"], a["sB"], a["C"], a["M"], a["N"], a["K"], mode, None)
    assert call(mode=7) == _abi.FP8_ERR_MODE
    assert call(mode=-1) == _abi.FP8_ERR_MODE
    for bad in (dict(N=12), dict(K=24), dict(M=-1), dict(N=-8), dict(K=-16), dict(M=1 << 30), dict(N=1 << 30),
                dict(K=1 << 30)):
        assert call(**bad) == _abi.FP8_ERR_SHAPE, bad
    for name in ("A", "sA", "B", "sB", "C"):
        assert call(**{name: 0}) == _abi.FP8_ERR_NULL, name
        assert call(**{name: 2 if name[0] == "s" else 8}) == _abi.FP8_ERR_ALIGN, name
    assert call(A=0, sA=0, B=0, sB=0, C=0, M=0) == _abi.FP8_OK
    assert call(A=0, sA=0, B=0, sB=0, C=0, N=0) == _abi.FP8_OK
    assert lib.fp8_gemm_block128(0, 0, 0, 0, 0, 64, 60, 64, None) == _abi.FP8_ERR_SHAPE


def test_experts_refusals(lib):
    def call(mode=0, **kw):
        a = dict(A=16, sA=16, B=16, sB=16, C=16, off=16, T=64, N=64, K=64, E=4)
        a.update(kw)
        return lib.fp8_gemm_experts_ex(a["A"], a["sA"], a["B"], a["sB"], a["C"], a["off"], a["T"], a["N"], a["K"],
                                       a["E"], mode, None)
    assert call(mode=3) == _abi.FP8_ERR_MODE
    for bad in (dict(N=12), dict(K=24), dict(T=-1), dict(E=-1), dict(E=_abi.FP8_MAX_EXPERTS + 1), dict(K=0),
                dict(T=1 << 30)):
        assert call(**bad) == _abi.FP8_ERR_SHAPE, bad
    for name in ("A", "sA", "B", "sB", "C", "off"):
        assert call(**{name: 0}) == _abi.FP8_ERR_NULL, name
        assert call(**{name: 8 if name in "ABC" else 2}) == _abi.FP8_ERR_ALIGN, name
    for none in (dict(T=0), dict(N=0), dict(E=0)):
        assert call(A=0, sA=0, B=0, sB=0, C=0, off=0, **none) in (_abi.FP8_OK, _abi.FP8_ERR_NULL)
    assert call(T=0) == _abi.FP8_OK and call(E=0) == _abi.FP8_OK
    assert lib.fp8_gemm_experts(0, 0, 0, 0, 0, 0, 64, 60, 64, 4, None) == _abi.FP8_ERR_SHAPE


def test_quantizer_refusals(lib):
    def call(**kw):
        a = dict(x=16, ldx=64, x_rows=64, rows=0, q=16, s=16, M=64, K=64, flags=0)
        a.update(kw)
        return lib.fp8_quantize_tokens(a["x"], a["ldx"], a["x_rows"], a["rows"], a["q"], a["s"], a["M"], a["K"],
                                       a["flags"], None)
    for bad in (dict(K=24), dict(ldx=56), dict(ldx=68), dict(M=-1), dict(K=-16), dict(x_rows=-1), dict(x_rows=63),
                dict(M=1 << 30, x_rows=1 << 30)):
        assert call(**bad) == _abi.FP8_ERR_SHAPE, bad
    assert call(flags=2) == _abi.FP8_ERR_MODE
    for name in ("x", "q", "s"):
        assert call(**{name: 0}) == _abi.FP8_ERR_NULL, name
    for bad in (dict(x=8), dict(q=8), dict(s=2), dict(rows=2)):
        assert call(**bad) == _abi.FP8_ERR_ALIGN, bad
    assert call(M=0) == _abi.FP8_OK
    gated = lambda **kw: lib.fp8_swiglu_quantize_tokens(16, kw.get("ldx", 128), 16, 16, kw.get("M", 64),   # noqa: E731
                                                        kw.get("K", 64), kw.get("flags", 0), None)
    assert gated(ldx=120) == _abi.FP8_ERR_SHAPE and gated(K=40) == _abi.FP8_ERR_SHAPE
    assert gated(flags=4) == _abi.FP8_ERR_MODE and gated(M=0) == _abi.FP8_OK


def test_python_refusals():
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype)   # noqa: E731
    A, sA, B, sB, C = z(4, 256), z(4, 2, dtype=torch.float32), z(136, 256), z(2, 2, dtype=torch.float32), \
        z(4, 136, dtype=torch.bfloat16)
    for bad in ((A, sA[:, :1], B, sB, C), (A, sA, B, sB[:1], C), (A, sA, B[:, :128], sB, C), (A, sA, B, sB, C[:3])):
        with pytest.raises(ValueError):
            bs.fp8_gemm_block128(*bad)
    with pytest.raises(ValueError, match="contiguous"):
        bs.fp8_gemm_block128(z(256, 4).T, sA, B, sB, C)
    with pytest.raises(ValueError, match="type"):
        bs.fp8_gemm_block128(A, sA, B, sB, C.float())
    with pytest.raises(ValueError, match="type"):
        bs.fp8_gemm_block128(A.to(torch.bfloat16), sA, B, sB, C)
    B3, sB3 = z(3, 136, 256), z(3, 2, 2, dtype=torch.float32)
    with pytest.raises(ValueError):
        bs.fp8_gemm_experts(A, sA, B3, sB3, C, z(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="type"):
        bs.fp8_gemm_experts(A, sA, B3, sB3, C, z(4, dtype=torch.int64))
    x = z(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bs.fp8_quantize_tokens(x, q=z(4, 128))
    with pytest.raises(ValueError, match="type"):
        bs.fp8_quantize_tokens(x.float())
    with pytest.raises(ValueError, match="type"):
        bs.fp8_quantize_tokens(x, rows=z(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        bs.fp8_quantize_tokens(z(256, 4, dtype=torch.bfloat16).T)
    with pytest.raises(ValueError, match="type"):
        bs.fp8_quantize_tokens(x.to(torch.float16))
    for call in (lambda: bs.fp8_gemm_block128(A, sA, B, sB, C), lambda: bs.fp8_quantize_tokens(x),
                 lambda: bs.fp8_gemm_experts(A, sA, B3, sB3, C, z(4, dtype=torch.int32)),
                 lambda: bs.fp8_swiglu_quantize_tokens(x)):
        with pytest.raises(ValueError, match="GPU"):   # host tensors
            call()
    with pytest.raises(ValueError):
        bs.fp8_swiglu_quantize_tokens(z(4, 33, dtype=torch.bfloat16))
