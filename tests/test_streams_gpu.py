"""Calls on another stream than the current one: outputs that a call allocates belong to the
stream that writes them, and a call runs after what its stream was given before it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bs():
    import block_scaled_fp8_sm_gb300 as mod
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    mod.library()
    return mod


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["fp8_quantize_tokens", "fp8_swiglu_quantize_tokens", "fp8_quantize_blocks"])
def test_outputs_belong_to_the_stream_that_writes_them(bs, name, handle):
    """Memory freed on the current stream may still be in use by its queued work: a call on
    another stream must not be given it."""
    M, K = 4096, 4096
    x = torch.randn(M, 2 * K if "swiglu" in name else K, device=DEV).to(torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = torch.empty(M, K, dtype=torch.uint8, device=DEV)
    where = freed.data_ptr()
    del freed
    q, s = getattr(bs, name)(x, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert q.data_ptr() != where
    want = getattr(bs, name)(x)
    torch.cuda.synchronize()
    assert want[0].data_ptr() == where   # on the current stream the block is free
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])
