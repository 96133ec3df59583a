"""The router against its definition in 64 bits: whole numbers exactly, weights in fp32."""
import math

import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from tests import _moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_sm_gb300 import build
    build.build()


def logits(T, E, seed, dtype=torch.float32, closed=0.0, empty=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * 3
    if closed:
        x[torch.rand(T, E, generator=g) < closed] = -math.inf
        x[torch.rand(T, generator=g) < empty] = -math.inf
    return x.to(dtype)


def check(x, top, out=None, got=None, **kw):
    res = bs.fp8_moe_route(x.cuda(), top, out=out, **kw) if got is None else got
    kw.pop("workspace", None), kw.pop("stream", None)
    w, ids, offsets, rows, places, tol = _moe.route(x, top, **kw)
    torch.cuda.synchronize()
    gw, gi, go, gr, gp = (t.cpu() for t in res)
    assert torch.equal(gi.long(), ids)
    assert torch.equal(go.long(), offsets) and torch.equal(gr.long(), rows) and torch.equal(gp.long(), places)
    err = (gw.double() - w).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    return res


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 700])
@pytest.mark.parametrize("E,top", [(1, 1), (2, 2), (31, 3), (32, 32), (33, 8), (64, 4), (96, 6), (250, 8), (256, 8),
                                   (300, 5), (520, 32), (1024, 7)])
def test_sizes(T, E, top):
    check(logits(T, E, T * 31 + E), top)


@pytest.mark.parametrize("T", [1, 40, 333])
@pytest.mark.parametrize("E,top", [(2, 1), (40, 3), (64, 8), (128, 8), (256, 8), (512, 6), (1001, 9)])
def test_bf16_with_ties(T, E, top):
    x = logits(T, E, T + E, torch.bfloat16)
    check(x, top)
    check((x * 2).round(), top)   # many equal logits


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,top", [(5, 16, 4), (130, 200, 8)])
def test_weights(T, E, top, sigmoid, renormalize):
    check(logits(T, E, 3), top, sigmoid=sigmoid, renormalize=renormalize, scale=2.5)
    check(logits(T, E, 4, closed=0.5, empty=0.2), top, sigmoid=sigmoid, renormalize=renormalize)
    check(logits(T, E, 5) * 60, top, sigmoid=sigmoid, renormalize=renormalize)     # far apart
    check(logits(T, E, 6) - 200, top, sigmoid=sigmoid, renormalize=renormalize)    # sigmoids below fp32's range


@pytest.mark.parametrize("T", [4, 90])
def test_closed_experts_and_empty_rows(T):
    x = logits(T, 48, 9, closed=0.9, empty=0.3)
    x[0] = -math.inf
    x[1] = float("nan")
    x[2, :] = -math.inf
    x[2, 17] = torch.finfo(torch.float32).min   # the type's lowest value is open
    w, ids, offsets, rows, places = check(x, 6)
    assert ids[0].tolist() == [-1] * 6 and not w[0].any() and ids[2].tolist() == [17] + [-1] * 5
    assert float(w[2, 0]) == 1.0 and int(offsets[-1]) == int((ids >= 0).sum())
    assert bool((rows[int(offsets[-1]):] == -1).all())
    check(torch.full((T, 48), -math.inf), 6)


def test_special_values():
    x = torch.zeros(6, 8)
    x[0, 3] = -0.0                       # -0 and +0 are equal: the lower expert first
    x[1, 2], x[1, 6] = math.inf, math.inf
    x[2, 4] = float("nan")
    x[3] = torch.finfo(torch.float32).max
    x[4] = torch.arange(8) * 1e-42       # subnormal numbers keep their order
    x[5] = -torch.arange(8) * 1e38
    for sigmoid in (False, True):
        w, ids, *_ = check(x, 3, sigmoid=sigmoid)
        assert ids[0].tolist() == [0, 1, 2] and ids[1].tolist()[:2] == [2, 6] and bool(w.isfinite().all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,ld,at", [(64, 72, 0), (64, 67, 1), (256, 264, 4), (256, 300, 2), (12, 13, 1)])
def test_strided_rows(E, ld, at, dtype):
    x = logits(70, ld, ld, dtype)
    on = x.cuda()[:, at:at + E] if at + E <= ld else x.cuda()[:, :E]
    host = x[:, at:at + E] if at + E <= ld else x[:, :E]
    for T in (1, 9, 70):
        check(host[:T], 4, got=bs.fp8_moe_route(on[:T], 4))


@pytest.mark.parametrize("T,E,top", [(16001, 256, 8), (40000, 64, 4), (20000, 1024, 2)])
def test_long(T, E, top):
    check(logits(T, E, T, closed=0.3, empty=0.01), top, sigmoid=True)


def test_without_an_order():
    x = logits(500, 64, 1)
    w, ids = bs.fp8_moe_route(x.cuda(), 4, order=False)
    ref = _moe.route(x, 4)
    assert torch.equal(ids.cpu().long(), ref[1])
    assert bool(((w.cpu().double() - ref[0]).abs() <= ref[5]).all())


def test_no_tokens():
    w, ids, offsets, rows, places = bs.fp8_moe_route(torch.empty(0, 16, device="cuda"), 4)
    assert w.shape == (0, 4) and rows.shape == (0,) and offsets.tolist() == [0] * 17


@pytest.mark.parametrize("T", [12, 900])
def test_outputs_are_written_in_full_each_time(T):
    first = bs.fp8_moe_route(logits(T, 40, 1).cuda(), 5)
    space = torch.full((bs.fp8_moe_route_workspace_bytes(T, 40, 5),), 255, dtype=torch.uint8, device="cuda")
    for t in first:
        t.fill_(99)
    for seed in (2, 3):
        assert check(logits(T, 40, seed, closed=0.4, empty=0.1), 5, out=first, workspace=space) is first


@pytest.mark.parametrize("T", [20, 3000])
def test_replays_in_a_graph_and_on_another_stream(T):
    x = logits(T, 64, 1)
    on = x.cuda()
    out = bs.fp8_moe_route(on, 4)
    space = torch.empty(bs.fp8_moe_route_workspace_bytes(T, 64, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.fp8_moe_route(on, 4, out=out, workspace=space)
    for seed in (2, 3):
        x = logits(T, 64, seed, closed=0.2)
        on.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        check(x, 4, got=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(x, 4, got=bs.fp8_moe_route(on, 4, stream=side))
    del graph
