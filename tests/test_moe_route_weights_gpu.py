"""The router's weights where fp32 has no excuse: equal logits, whose quotient is 1 / n."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_sm_gb300 import build
    build.build()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("E", [32, 200])
def test_equal_logits(T, E, sigmoid):
    """Every part is exact (exp(0) = 1, a sigmoid of 1/2, sums of them), so that the weight is
    1 / n rounded once, of the chosen or of all open experts."""
    for top in range(1, 33):
        x = torch.zeros(T, E, device="cuda")
        w, ids = bs.fp8_moe_route(x, top, sigmoid=sigmoid, order=False)
        assert torch.equal(w.cpu(), torch.ones(T, top) / torch.full((T, top), float(top))), top
        assert torch.equal(ids.cpu(), torch.arange(top, dtype=torch.int32).expand(T, top))
        if not sigmoid:
            x[:, top:] = -float("inf")
            w, _ = bs.fp8_moe_route(x, 1, renormalize=False, order=False)
            assert torch.equal(w.cpu(), torch.ones(T, 1) / torch.full((T, 1), float(top))), top
