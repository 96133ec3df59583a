"""The layer's activation between its products, where sixteen of its values are far below the
others of their 128: they are kept to 2^-22 of the largest, whichever form serves the call."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from tests._fused import values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_sm_gb300 import build
    build.build()


def codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8).cuda()


# the form for few tokens (one eight, several), tiles for few tokens and for more
@pytest.mark.parametrize("T,top,E,H,I", [(3, 1, 2, 272, 272), (21, 1, 2, 528, 400), (7, 3, 32, 2048, 1552),
                                         (9, 8, 20, 2064, 1040), (21, 4, 6, 2064, 2064), (40, 1, 2, 2064, 2064)])
def test_small_groups(T, top, E, H, I):   # noqa: E741
    g = torch.Generator().manual_seed(T + I)
    # column i of h is silu(gate x0) (up x0): the groups of sixteen columns are 2^12 and more, and 2^-17
    # to 2^-23 of that, in turn; row n of down reads the columns of group n mod 8 alone
    group = torch.arange(I) // 16 % 8
    gate = torch.where(group == 0, 16.0, 0.25)
    up = torch.where(group == 0, torch.tensor(256.0), 2.0 ** (-1.0 - group))
    gate_up = torch.zeros(E, 2 * I, H)
    gate_up[:, :I, 0], gate_up[:, I:, 0] = gate, up
    down = torch.where(torch.arange(H)[:, None] % 8 == group, torch.rand(E, H, I, generator=g) + 0.5, torch.zeros(1))
    gate_up, down = codes(gate_up), codes(down)
    hb, ib = -(-H // 128), -(-I // 128)
    s_gate_up, s_down = torch.ones(E, -(-2 * I // 128), hb, device="cuda"), torch.ones(E, hb, ib, device="cuda")
    x = torch.randn(T, H, generator=g)
    x[:, 0] = torch.rand(T, generator=g) + 1.0
    x = x.to(torch.bfloat16).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(T)]).to(torch.int32).cuda()
    w = (torch.rand(T, top, generator=g) + 0.5).cuda()
    out = bs.fp8_moe_layer(x, w, ids, gate_up, s_gate_up, down, s_down)
    want, bound = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    x0 = x[:, :1].double()
    y = x0 * gate.double().cuda()
    h = y * torch.sigmoid(y) * (x0 * up.double().cuda())
    largest = torch.zeros(T, ib * 128, dtype=torch.float64, device="cuda")
    largest[:, :I] = h.abs()
    largest = largest.view(T, ib, 128).amax(2).repeat_interleave(128, 1)[:, :I]
    # h: 11 bits, 2^-13 for the gate, and 2^-22 of the largest of the 128; 1e-5 for the fp32 sums
    dh = (2.0 ** -11 + 2.0 ** -13 + 1e-5) * h.abs() + 2.0 ** -22 * largest
    for e in range(E):
        D = values(down[e], s_down[e], 128)
        f = torch.where(ids == e, w, torch.zeros_like(w)).double().sum(1, keepdim=True)
        want += f * (h @ D.T)
        bound += f * (dh @ D.T)
    bound += 2.0 ** -8 * want.abs()
    err = (out.double() - want).abs()
    worst = (err / bound).amax(0).cpu().view(-1, 8).amax(0)   # of the rows that read group 0, 1, ...
    assert bool((worst <= 1).all()), worst.tolist()
