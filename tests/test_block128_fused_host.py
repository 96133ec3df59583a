"""Refusals of the fused product (no GPU: each comes before a device is touched)."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from block_scaled_fp8_sm_gb300 import _abi


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    return bs.library()


def test_refusals(lib):
    def call(**kw):
        a = dict(A=16, sA=16, B=16, sB=16, bias=16, type=0, act=0, R=16, C=16, M=64, N=64, K=64, mode=0)
        a.update(kw)
        return lib.fp8_gemm_block128_fused(a["A"], a["sA"], a["B"], a["sB"], a["bias"], a["type"], a["act"], a["R"],
                                           a["C"], a["M"], a["N"], a["K"], a["mode"], None)
    for bad in (dict(mode=7), dict(mode=-1), dict(type=2), dict(type=-1), dict(act=5), dict(act=-1)):
        assert call(**bad) == _abi.FP8_ERR_MODE, bad
    for bad in (dict(N=12), dict(K=24), dict(M=-1), dict(N=-8), dict(K=-16), dict(M=1 << 30), dict(N=1 << 30),
                dict(K=1 << 30)):
        assert call(**bad) == _abi.FP8_ERR_SHAPE, bad
    for name in ("A", "sA", "B", "sB", "C"):
        assert call(**{name: 0}) == _abi.FP8_ERR_NULL, name
        assert call(**{name: 2 if name[0] == "s" else 8}) == _abi.FP8_ERR_ALIGN, name
    for name in ("bias", "R"):
        assert call(**{name: 8}) == _abi.FP8_ERR_ALIGN, name
    assert call(M=0) == _abi.FP8_OK and call(N=0) == _abi.FP8_OK
    assert call(M=0, act=9) == _abi.FP8_ERR_MODE   # wrong choices are told without work, too


def test_python_refusals():
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype)   # noqa: E731
    f32, bf16 = torch.float32, torch.bfloat16
    ops = (z(4, 256), z(4, 2, dtype=f32), z(136, 256), z(2, 2, dtype=f32), z(4, 136, dtype=bf16))
    for i, bad in ((1, ops[1][:, :1]), (2, ops[2][:, :128]), (3, ops[3][:1]), (4, ops[4][:3])):
        with pytest.raises(ValueError, match="shapes"):
            bs.fp8_gemm_block128_fused(*ops[:i], bad, *ops[i + 1:])
    for named in (dict(bias=z(135, dtype=f32)), dict(bias=z(1, 136, dtype=f32)), dict(residual=z(4, 128, dtype=bf16)),
                  dict(residual=z(136, dtype=bf16))):
        with pytest.raises(ValueError, match="shapes"):
            bs.fp8_gemm_block128_fused(*ops, **named)
    for named in (dict(bias=z(136, dtype=torch.float16)), dict(bias=z(136, dtype=torch.float64)),
                  dict(residual=z(4, 136, dtype=f32))):
        with pytest.raises(ValueError, match="type"):
            bs.fp8_gemm_block128_fused(*ops, **named)
    for named in ({}, dict(bias=z(272, dtype=f32)[::2]), dict(residual=z(136, 4, dtype=bf16).T)):
        with pytest.raises(ValueError, match="contiguous"):
            bs.fp8_gemm_block128_fused(*ops, **named)
