"""The 128-granular calls launch on the current device: tensors of another device, or of
several, are refused before anything is launched (stand-ins for the tensors and the library:
no second device is needed)."""
import types

import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs


class On:
    """A tensor that says it is on CUDA device `device`."""
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
    fake = types.SimpleNamespace(codes=frozenset((torch.uint8, torch.float8_e4m3fn)), f32=torch.float32,
                                 bf16=torch.bfloat16, i32=torch.int32, stream=lambda dev: 1000 + dev,
                                 device=lambda: current[0], block128=launch, experts=launch, quantize=launch,
                                 swiglu=launch)
    monkeypatch.setattr(bs._Calls, "loaded", fake)
    return made, lambda d: current.__setitem__(0, d)


def z(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype)


F, H, I = torch.float32, torch.bfloat16, torch.int32
CALLS = {
    "fp8_gemm_block128": ((z(4, 256), z(4, 2, dtype=F), z(136, 256), z(2, 2, dtype=F), z(4, 136, dtype=H)), {}),
    "fp8_gemm_experts": ((z(4, 256), z(4, 2, dtype=F), z(3, 136, 256), z(3, 2, 2, dtype=F), z(4, 136, dtype=H),
                          z(4, dtype=I)), {}),
    "fp8_quantize_tokens": ((z(4, 256, dtype=H), z(4, 256), z(4, 2, dtype=F)), {"rows": z(4, dtype=I)}),
    "fp8_swiglu_quantize_tokens": ((z(4, 512, dtype=H), z(4, 256), z(4, 2, dtype=F)), {}),
}


@pytest.mark.parametrize("name", CALLS)
def test_other_devices_are_refused(calls, name):
    made, set_current = calls
    args, named = CALLS[name]
    call = getattr(bs, name)

    def run(device, odd=None, odd_device=None):
        a = [On(t, odd_device if i == odd else device) for i, t in enumerate(args)]
        k = {n: On(t, odd_device if n == odd else device) for n, t in named.items()}
        return call(*a, **k)

    run(0)
    assert len(made) == 1 and made[0][-1] == 1000   # the stream of the current device
    for odd in list(range(len(args))) + list(named):   # one operand elsewhere
        for device, elsewhere in ((0, 1), (1, 0)):
            with pytest.raises(ValueError, match="device"):
                run(device, odd, elsewhere)
    with pytest.raises(ValueError, match="current device 0"):
        run(1)                                          # all of them elsewhere
    assert len(made) == 1, "a call with tensors of another device was launched"
    set_current(1)
    run(1)
    assert len(made) == 2 and made[1][-1] == 1001
