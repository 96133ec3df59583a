"""Refusals of the router and of the layer (no GPU: each comes before a device is touched),
and how their kernels read memory."""
import os
import re
import types

import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from block_scaled_fp8_sm_gb300 import _abi

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp8_sm_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    return bs.library()


def test_route_refusals(lib):
    def call(**kw):
        a = dict(logits=16, ld=64, type=0, T=200, E=64, top=4, flags=0, scale=1.0, weights=16, ids=16, offsets=16,
                 rows=16, places=16, space=16, bytes=1 << 20)
        a.update(kw)
        return lib.fp8_moe_route(a["logits"], a["ld"], a["type"], a["T"], a["E"], a["top"], a["flags"], a["scale"],
                                 a["weights"], a["ids"], a["offsets"], a["rows"], a["places"], a["space"],
                                 a["bytes"], None)
    for bad in (dict(type=2), dict(type=-1), dict(flags=4), dict(flags=-1)):
        assert call(**bad) == _abi.FP8_ERR_MODE, bad
    for bad in (dict(T=-1), dict(T=1 << 30), dict(T=1 << 29), dict(E=0), dict(E=1025, ld=1025), dict(top=0),
                dict(top=33), dict(top=5, E=4), dict(ld=63), dict(ld=1 << 31), dict(bytes=16), dict(bytes=-1)):
        assert call(**bad) == _abi.FP8_ERR_SHAPE, bad
    for name in ("logits", "weights", "ids", "rows", "places", "space"):
        assert call(**{name: 0}) == _abi.FP8_ERR_NULL, name
    assert call(offsets=0) == _abi.FP8_ERR_NULL   # rows without offsets
    for name in ("logits", "weights", "ids", "offsets", "rows", "places", "space"):
        assert call(**{name: 18}) == _abi.FP8_ERR_ALIGN, name
    assert call(T=0, offsets=0, rows=0, places=0) == _abi.FP8_OK
    assert bs.fp8_moe_route_workspace_bytes(1, 64, 4) == 0
    assert bs.fp8_moe_route_workspace_bytes(16384, 64, 4) > 0
    for bad in ((-1, 64, 4), (10, 0, 1), (10, 64, 0), (10, 4, 5)):
        assert bs.fp8_moe_route_workspace_bytes(*bad) == 0


def test_layer_refusals(lib):
    def call(**kw):
        a = dict(x=16, w=16, ids=16, W1=16, s1=16, W2=16, s2=16, out=16, T=8, top=4, E=32, H=256, I=128, space=16,
                 bytes=1 << 23)
        a.update(kw)
        return lib.fp8_moe_layer(a["x"], a["w"], a["ids"], a["W1"], a["s1"], a["W2"], a["s2"], a["out"], a["T"],
                                 a["top"], a["E"], a["H"], a["I"], a["space"], a["bytes"], None)
    for bad in (dict(T=-1), dict(T=65), dict(top=0), dict(top=33), dict(E=-1), dict(E=1025), dict(H=-16),
                dict(H=24), dict(H=1 << 30), dict(I=24), dict(I=-16), dict(I=1 << 30), dict(bytes=100), dict(bytes=-1)):
        assert call(**bad) == _abi.FP8_ERR_SHAPE, bad
    for name in ("x", "w", "ids", "W1", "s1", "W2", "s2", "out", "space"):
        assert call(**{name: 0}) == _abi.FP8_ERR_NULL, name
        wide = name in ("x", "W1", "W2", "out", "space")
        assert call(**{name: 8 if wide else 18}) == _abi.FP8_ERR_ALIGN, name
    assert call(T=0) == _abi.FP8_OK and call(H=0) == _abi.FP8_OK
    assert bs.fp8_moe_layer_workspace_bytes(8, 4, 128) >= 8 * 4 * (256 + 32)   # h and its scales, and more
    for bad in ((65, 4, 128), (8, 0, 128), (8, 4, 24), (-1, 4, 128)):
        assert bs.fp8_moe_layer_workspace_bytes(*bad) == 0


def z(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype)


F, H, I32 = torch.float32, torch.bfloat16, torch.int32


def test_python_route_refusals():
    x = z(4, 64, dtype=F)
    out = (z(4, 2, dtype=F), z(4, 2, dtype=I32), z(65, dtype=I32), z(8, dtype=I32), z(4, 2, dtype=I32))
    for i in range(5):
        with pytest.raises(ValueError, match="must be"):
            bs.fp8_moe_route(x, 2, out=out[:i] + (out[i][:1],) + out[i + 1:])
    with pytest.raises(ValueError, match="must be"):
        bs.fp8_moe_route(x, 2, out=out[:2])
    with pytest.raises(ValueError, match="must be"):
        bs.fp8_moe_route(x, 2, out=out, order=False)
    with pytest.raises(ValueError, match="type"):
        bs.fp8_moe_route(x.half(), 2)
    with pytest.raises(ValueError, match="type"):
        bs.fp8_moe_route(x, 2, out=out[:1] + (out[1].long(),) + out[2:])
    with pytest.raises(ValueError, match="contiguous"):
        bs.fp8_moe_route(z(64, 4, dtype=F).T, 2)
    with pytest.raises(ValueError, match="GPU"):
        bs.fp8_moe_route(x, 2)


def test_python_layer_refusals():
    args = [z(4, 256, dtype=H), z(4, 2, dtype=F), z(4, 2, dtype=I32), z(3, 160, 256), z(3, 2, 2, dtype=F),
            z(3, 256, 80), z(3, 2, 1, dtype=F), z(4, 256, dtype=H)]
    cut = {0: args[0][:, :240], 1: args[1][:3], 2: args[2][:, :1], 3: args[3][:, :159], 4: args[4][:, :1],
           5: args[5][:2], 6: args[6][:, :1], 7: args[7][:3]}
    for i, bad in cut.items():
        with pytest.raises(ValueError, match="shapes"):
            bs.fp8_moe_layer(*args[:i], bad, *args[i + 1:])
    with pytest.raises(ValueError, match="65 tokens"):
        bs.fp8_moe_layer(z(65, 256, dtype=H), z(65, 2, dtype=F), z(65, 2, dtype=I32), *args[3:7])
    for i, kind in ((0, F), (1, H), (2, torch.int64), (3, torch.int8), (4, H), (5, torch.int8), (6, H), (7, F)):
        with pytest.raises(ValueError, match="type"):
            bs.fp8_moe_layer(*args[:i], args[i].to(kind), *args[i + 1:])
    with pytest.raises(ValueError, match="contiguous"):
        bs.fp8_moe_layer(z(256, 4, dtype=H).T, *args[1:])
    with pytest.raises(ValueError, match="GPU"):
        bs.fp8_moe_layer(*args)


class On:
    """A tensor that says it is on CUDA device `device` (no second device is needed)."""
    is_cuda = True

    def __init__(self, t, device):
        self._t, self._device = t, device
        self.shape, self.dtype, self.device = t.shape, t.dtype, torch.device("cuda", device)

    def get_device(self):
        return self._device

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def calls(monkeypatch):
    """(list of launches, setter of the current device)"""
    made, current = [], [0]
    launch = lambda *a: made.append(a) or 0   # noqa: E731
    fake = types.SimpleNamespace(codes=frozenset((torch.uint8, torch.float8_e4m3fn)), f32=F, bf16=H, i32=I32,
                                 floats=frozenset((F, H)), stream=lambda dev: 1000 + dev, device=lambda: current[0],
                                 fused=launch, route=launch, layer=launch)
    monkeypatch.setattr(bs._Calls, "loaded", fake)
    return made, lambda d: current.__setitem__(0, d)


def fused(A, sA, B, sB, C, bias, R):
    return bs.fp8_gemm_block128_fused(A, sA, B, sB, C, bias=bias, residual=R)


def route(logits, weights, ids, offsets, rows, places, space):
    return bs.fp8_moe_route(logits, 2, out=(weights, ids, offsets, rows, places), workspace=space)


CALLS = {
    "fused": (fused, (z(4, 256), z(4, 2, dtype=F), z(136, 256), z(2, 2, dtype=F), z(4, 136, dtype=H), z(136, dtype=F),
                      z(4, 136, dtype=H))),
    "route": (route, (z(4, 64, dtype=F), z(4, 2, dtype=F), z(4, 2, dtype=I32), z(65, dtype=I32), z(8, dtype=I32),
                      z(4, 2, dtype=I32), z(64))),
    "layer": (bs.fp8_moe_layer, (z(4, 256, dtype=H), z(4, 2, dtype=F), z(4, 2, dtype=I32), z(3, 160, 256),
                                 z(3, 2, 2, dtype=F), z(3, 256, 80), z(3, 2, 1, dtype=F), z(4, 256, dtype=H), z(4096))),
}


@pytest.mark.parametrize("name", CALLS)
def test_other_devices_are_refused(calls, name):
    made, set_current = calls
    call, args = CALLS[name]

    def run(device, odd=None, odd_device=None):
        return call(*[On(t, odd_device if i == odd else device) for i, t in enumerate(args)])

    run(0)
    assert len(made) == 1 and made[0][-1] == 1000   # the stream of the current device
    for odd in range(len(args)):   # one tensor elsewhere
        for device, elsewhere in ((0, 1), (1, 0)):
            with pytest.raises(ValueError, match="device"):
                run(device, odd, elsewhere)
    with pytest.raises(ValueError, match="current device 0"):
        run(1)
    assert len(made) == 1, "a call with tensors of another device was launched"
    set_current(1)
    run(1)
    assert len(made) == 2 and made[1][-1] == 1001


@pytest.mark.parametrize("name", ["moe_layer.cuh", "moe_tile.cuh", "moe_route.cuh", "moe_api.cu", "epilogue.cuh", "host.h"])
def test_no_noncoherent_load(name):
    """Kernels that may start while the one before still writes read with ordinary loads."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\w*|ld\.global\.nc\S*|__restrict__", code)
