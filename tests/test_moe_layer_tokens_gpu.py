"""The mixture-of-experts layer for a few tokens against 64 bits, and the routed chain of
operators as a program runs it."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from tests import _moe
from tests._fused import values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_sm_gb300 import build
    build.build()


def compare(out, ref, bound, what=""):
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), f"{what}: worst {float((err / bound).max()):.3f} of the bound"


# T, top, E, H, I: one token, one expert, blocks that end early, sizes below a block, eights of
# tokens that are full and not, fewer blocks of K than warps and more (small weights)
SIZES = [(1, 1, 1, 16, 16), (1, 4, 32, 2048, 1024), (3, 8, 64, 512, 272), (8, 2, 4, 1040, 400), (9, 3, 5, 144, 2064),
         (19, 3, 16, 2064, 1040), (64, 8, 16, 528, 256), (64, 2, 2, 272, 48), (33, 32, 40, 256, 128),
         (64, 1, 1024, 64, 32), (17, 1, 1, 4112, 1296), (16, 2, 3, 144, 80), (25, 4, 5, 400, 1040), (32, 8, 9, 1040, 144),
         (57, 7, 8, 272, 2064), (48, 1, 2, 16, 16),
         (64, 4, 4, 4096, 1024), (40, 8, 12, 2048, 2048)]

# large weights, which tiles read: one, two, four and eight groups of eight tokens of an expert, one
# row of tiles, tiles and blocks that end early, many experts, every pair of a token
TILES = [(9, 8, 20, 2064, 1040), (12, 8, 30, 2064, 1040), (33, 32, 40, 1040, 528), (64, 32, 1024, 256, 272),
         (17, 1, 1, 4112, 4112), (48, 1, 2, 4112, 2064), (57, 7, 8, 528, 4112), (25, 4, 5, 1040, 4112),
         (30, 4, 48, 144, 5136), (30, 4, 48, 5136, 144), (64, 8, 256, 528, 272), (16, 2, 40, 1040, 2064)]


@pytest.mark.parametrize("T,top,E,H,I", SIZES + TILES)
def test_sizes(T, top, E, H, I):   # noqa: E741
    layer = _moe.Layer(E, H, I, T + H)
    x, w, ids = _moe.inputs(T, top, E, H, I)
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    bs.fp8_moe_layer(x, w, ids, *layer.weights, out)
    compare(out, *layer.reference(x, w, ids), f"{T} {top} {E} {H} {I}")


@pytest.mark.parametrize("T,H,I", [(2, 272, 144), (8, 272, 144), (21, 272, 144), (21, 2064, 2064)])
def test_padding_and_repeated_experts(T, H, I):   # noqa: E741
    layer = _moe.Layer(6, H, I, 3)
    x, w, ids = _moe.inputs(T, 4, 6, H, 5)
    ids[0] = -1                                           # a token without any expert
    ids[1] = torch.tensor([2, 2, -1, 2])                  # one expert three times
    ids[T - 1] = torch.tensor([5, 6, -7, 2 ** 31 - 1])    # numbers that no expert has
    w[T - 1, 1:] = float("nan")                           # their weights take no part
    x[0] = float("inf")                                   # nor do rows without experts
    keep = torch.where((ids >= 0) & (ids < 6), w, torch.zeros_like(w))
    out = bs.fp8_moe_layer(x, w, ids, *layer.weights)
    ref, bound = layer.reference(torch.where(x.isfinite(), x, torch.zeros_like(x)), keep, ids)
    compare(out, ref, bound)
    assert not out[0].any()


# weights that tiles read faster, however few the tokens are
@pytest.mark.parametrize("T,top,E,H,I", [(1, 32, 32, 2064, 2064), (4, 8, 10, 2064, 2032), (7, 3, 32, 2048, 1552)])
def test_few_tokens_of_large_weights(T, top, E, H, I):   # noqa: E741
    layer = _moe.Layer(E, H, I, T + H)
    x, w, ids = _moe.inputs(T, top, E, H, I)
    if T > 1:
        ids[0] = -1                                      # a token without any expert
        ids[1, 1:] = ids[1, 0]                           # one expert only, several times
        ids[2, 0] = E
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    bs.fp8_moe_layer(x, w, ids, *layer.weights, out)
    ref, bound = layer.reference(x, w, ids)
    compare(out, ref, bound, f"{T} {top} {E} {H} {I}")
    for _ in range(5):
        assert torch.equal(bs.fp8_moe_layer(x, w, ids, *layer.weights), out)
    bs.fp8_moe_layer(x, w, torch.full_like(ids, -1), *layer.weights, out)
    assert not out.any()


# the form for few tokens, tiles for few tokens, several eights, tiles
@pytest.mark.parametrize("T,top,E,H,I", [(6, 3, 5, 272, 400), (4, 8, 10, 2064, 2032), (20, 2, 6, 528, 272),
                                         (20, 2, 6, 2064, 2064)])
def test_nan_and_infinity_stay_with_their_tokens(T, top, E, H, I):   # noqa: E741
    layer = _moe.Layer(E, H, I, 12)
    x, w, ids = _moe.inputs(T, top, E, H, 13)
    out = bs.fp8_moe_layer(x, w, ids, *layer.weights)
    x[1, 5], x[2, H - 1], w[T - 1, 0] = float("nan"), float("-inf"), float("nan")
    bad = bs.fp8_moe_layer(x, w, ids, *layer.weights)
    mine = torch.zeros(T, dtype=torch.bool, device="cuda")
    mine[1] = mine[2] = mine[T - 1] = True
    assert torch.equal(bad[~mine], out[~mine])
    assert not bool(bad[mine].isfinite().any())
    # a weight that is NaN spoils its row's results for the expert's tokens
    x, w, ids = _moe.inputs(T, top, E, H, 13)
    e = int(ids[0, 0])
    layer.down[e, 17, 3] = 0x7F
    bad = bs.fp8_moe_layer(x, w, ids, *layer.weights)
    mine = (ids == e).any(1)
    want = torch.zeros(T, H, dtype=torch.bool, device="cuda")
    want[mine, 17] = True
    assert torch.equal(bad.isnan(), want) and torch.equal(bad[~want], out[~want])
    layer.gate_up[e, 3, H - 1] = 0xFF
    assert torch.equal(bs.fp8_moe_layer(x, w, ids, *layer.weights).isnan().all(1), mine)


@pytest.mark.parametrize("T", [1, 5, 30])
def test_weights_past_32_bits(T):
    """Codes of more than 2^32 bytes, the last expert's at their end."""
    E, H, I = 300, 4096, 2048   # noqa: E741
    free = torch.cuda.mem_get_info()[0]
    if free < 20 << 30:
        pytest.skip("not enough memory")
    part = _moe.Layer(2, H, I, 14)
    gate_up = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device="cuda")
    down = torch.zeros(E, H, I, dtype=torch.uint8, device="cuda")
    s_gate_up, s_down = torch.zeros(E, 2 * I // 128, H // 128, device="cuda"), torch.zeros(E, H // 128, I // 128, device="cuda")
    gate_up[-2:], s_gate_up[-2:], down[-2:], s_down[-2:] = part.weights
    x, w, ids = _moe.inputs(T, 2, 2, H, 15)
    compare(bs.fp8_moe_layer(x, w, ids + E - 2, gate_up, s_gate_up, down, s_down), *part.reference(x, w, ids))


def test_no_expert_at_all():
    layer = _moe.Layer(3, 64, 32, 1)
    x, w, ids = _moe.inputs(5, 2, 3, 64, 1)
    assert not bs.fp8_moe_layer(x, w, ids.fill_(-1), *layer.weights, torch.ones_like(x)).any()
    none = torch.empty(0, 64, 64, dtype=torch.uint8, device="cuda")
    assert not bs.fp8_moe_layer(x, w, ids, none, torch.empty(0, 1, 1, device="cuda"), none[:, :, :32].contiguous(),
                                torch.empty(0, 1, 1, device="cuda"), torch.ones_like(x)).any()
    assert bs.fp8_moe_layer(x[:0], w[:0], ids[:0], *layer.weights).shape == (0, 64)


@pytest.mark.parametrize("T,top,E,H,I", [(8, 4, 8, 528, 400), (7, 8, 32, 256, 272)])
def test_a_tokens_bits_do_not_depend_on_the_others(T, top, E, H, I):   # noqa: E741
    layer = _moe.Layer(E, H, I, 8)
    x, w, ids = _moe.inputs(T, top, E, H, 9)
    out = bs.fp8_moe_layer(x, w, ids, *layer.weights)
    for part in (slice(0, 1), slice(3, 7), slice(5, T), slice(T - 1, T)):
        some = bs.fp8_moe_layer(x[part].contiguous(), w[part].contiguous(), ids[part].contiguous(), *layer.weights)
        assert torch.equal(some, out[part])
    turn = torch.arange(T - 1, -1, -1, device="cuda")
    assert torch.equal(bs.fp8_moe_layer(x[turn], w[turn], ids[turn], *layer.weights), out[turn])


@pytest.mark.parametrize("T,top,E,H,I", [(9, 3, 5, 144, 2064), (64, 8, 32, 256, 272), (30, 4, 8, 2064, 400),
                                         (30, 4, 8, 2064, 2064), (64, 8, 256, 528, 272)])
def test_calls_repeat_bit_for_bit(T, top, E, H, I):   # noqa: E741
    layer = _moe.Layer(E, H, I, 8)
    x, w, ids = _moe.inputs(T, top, E, H, 9)
    out = bs.fp8_moe_layer(x, w, ids, *layer.weights)
    for _ in range(20):
        assert torch.equal(bs.fp8_moe_layer(x, w, ids, *layer.weights), out)


@pytest.mark.parametrize("T,E,H,I", [(6, 4, 256, 128), (14, 4, 256, 128), (40, 4, 256, 128), (14, 8, 2048, 2064),
                                     (40, 8, 2048, 1040)])
def test_ranges(T, E, H, I):   # noqa: E741
    """Activations near the ends of bf16's range, one token beside another."""
    layer = _moe.Layer(E, H, I, 2)
    x, w, ids = _moe.inputs(T, 2, E, H, 4)
    x[1] *= 2.0 ** -100
    x[2] *= 2.0 ** 55
    x[3, :128] *= 2.0 ** -60
    x[4] = 0
    compare(bs.fp8_moe_layer(x, w, ids, *layer.weights), *layer.reference(x, w, ids))
    y = x.clone()
    y[1], y[2, 5] = float("nan"), float("inf")   # stay in their own rows
    a, b = (bs.fp8_moe_layer(v, w, ids, *layer.weights) for v in (x, y))
    assert torch.equal(a[[0] + list(range(3, T))], b[[0] + list(range(3, T))]) and not bool(b[1:3].isfinite().any())


def test_deep_gates():
    """Gates far below zero beside large up values: the product is still there (each in a
    block of its own: fp16 holds a block's values down to 2^-28 of the largest)."""
    T, H, I = 2, 256, 16   # noqa: E741
    one = torch.ones(1, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    gate_up = torch.zeros(1, 2 * I, H, dtype=torch.uint8, device="cuda")
    down = torch.zeros(1, H, I, dtype=torch.uint8, device="cuda")
    for i in range(I):
        gate_up[0, i, 0], gate_up[0, I + i, 128], down[0, i, i] = one, one, one
    s1, s2 = torch.ones(1, 1, 2, device="cuda"), torch.ones(1, 2, 1, device="cuda")
    for g, u in ((-95.0, 1e30), (-130.0, 2e37), (-60.0, -1e20), (90.0, 1e-30), (-1e30, 1e30), (2e38, 1.0)):
        x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        x[0, 0], x[0, 128] = g, u
        out = bs.fp8_moe_layer(x, torch.ones(T, 1, device="cuda"), torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                               gate_up, s1, down, s2)
        gd, ud = x[0, 0].double(), x[0, 128].double()
        want = gd * torch.sigmoid(gd) * ud
        # 2^-8 of the result's rounding and 2^-11 of h's; exp's argument is rounded by 2^-24 |g|
        assert abs(out[0, 3].double() - want) <= (2.0 ** -8 + 2.0 ** -10) * abs(want) + 1e-37, (g, u)
        assert not out[1].any() and not out[0, 16:].any()


@pytest.mark.parametrize("H,I", [(272, 144), (2064, 2064)])
def test_replays_in_a_graph_and_on_another_stream(H, I):   # noqa: E741
    layer = _moe.Layer(8, H, I, 3)
    T, top = 12, 3
    x, w, ids = _moe.inputs(T, top, 8, H, 1)
    out = torch.empty_like(x)
    space = torch.empty(bs.fp8_moe_layer_workspace_bytes(T, top, I), dtype=torch.uint8, device="cuda")
    bs.fp8_moe_layer(x, w, ids, *layer.weights, out, space)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.fp8_moe_layer(x, w, ids, *layer.weights, out, space)
    for seed in (2, 3):
        for old, new in zip((x, w, ids), _moe.inputs(T, top, 8, H, seed)):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        compare(out, *layer.reference(x, w, ids))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = bs.fp8_moe_layer(x, w, ids, *layer.weights, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    del graph


@pytest.mark.parametrize("T,top,E,H,I", [(5, 2, 8, 272, 144), (64, 4, 16, 512, 272), (40, 4, 16, 2048, 1040)])
def test_routed_chain(T, top, E, H, I):   # noqa: E741
    """Router, layer, and the same layer by the operators for many tokens, called as a
    program does, without a synchronization between them: the layer against 64 bits, the
    chain within the rounding of its FP8 activations."""
    layer = _moe.Layer(E, H, I, 5)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=g)
    logits[1] = -float("inf")   # a row of padding
    logits = logits.cuda()
    for _ in range(3):   # calls overlap at their ends
        w, ids, offsets, rows, places = bs.fp8_moe_route(logits, top)
        out = bs.fp8_moe_layer(x, w, ids, *layer.weights)
        A, sA = bs.fp8_quantize_tokens(x, rows=rows)
        h = torch.empty(T * top, 2 * I, dtype=torch.bfloat16, device="cuda")
        bs.fp8_gemm_experts(A, sA, layer.gate_up, layer.s_gate_up, h, offsets)
        A, sA = bs.fp8_swiglu_quantize_tokens(h)
        y = torch.empty(T * top, H, dtype=torch.bfloat16, device="cuda")
        bs.fp8_gemm_experts(A, sA, layer.down, layer.s_down, y, offsets)
        chain = (torch.where(places[:, :, None] >= 0, y[places.clamp(min=0).long()].float(), 0) * w[:, :, None]).sum(1)
    ref, bound = layer.reference(x, w, ids)
    compare(out, ref, bound)
    assert not out[1].any()
    # E4M3 is off by at most 2^-4 of a value, 2^-4 / sqrt(3) / 2 rms; three roundings that
    # the gate at most stretches by sqrt(2): 0.018 sqrt(1 + 2 + 1), and twice that is accepted
    assert float((chain - ref).norm() / ref.norm()) < 0.072
    assert bs.fp8_status_query() == 0


def test_reference_values_of_the_weights():
    """The layer of identity matrices is silu(x) * x of its own columns (no reference sum)."""
    H = I = 32   # noqa: E741
    eye = torch.eye(H, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.ones(1, 1, 1, device="cuda")
    x = torch.linspace(-6, 6, 4 * H).view(4, H).to(torch.bfloat16).cuda()
    out = bs.fp8_moe_layer(x, torch.ones(4, 1, device="cuda"), torch.zeros(4, 1, dtype=torch.int32, device="cuda"),
                           torch.cat([eye, eye])[None].contiguous(), s, eye[None].contiguous(), s)
    v = x.double()
    want = v * torch.sigmoid(v) * v
    assert bool(((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -30).all())
    assert torch.equal(values(eye, s[0], 128), torch.eye(H, dtype=torch.float64, device="cuda"))


@pytest.mark.parametrize("T,stage", [(12, 0), (12, 3), (40, 1)])
def test_withheld_stage_times_out_cleanly(T, stage):
    """Waits that run out are reported, the kernels return, and the next call is right."""
    layer = _moe.Layer(4, 2064, 2064, 6)
    x, w, ids = _moe.inputs(T, 3, 4, 2064, 7)
    space = torch.empty(bs.fp8_moe_layer_workspace_bytes(T, 3, 2064), dtype=torch.uint8, device="cuda")
    assert bs.fp8_status_query() == 0
    bs.fp8_debug_set(bs.FP8_DEBUG_WAIT_LIMIT_CYCLES, 20_000_000)   # ~10 ms
    bs.fp8_debug_set(bs.FP8_DEBUG_WITHHOLD_STAGE, stage)
    try:
        bs.fp8_moe_layer(x, w, ids, *layer.weights, workspace=space)
        torch.cuda.synchronize()
        assert bs.fp8_status_query() == bs._abi.FP8_ERR_TIMEOUT
    finally:
        bs.fp8_debug_set(bs.FP8_DEBUG_WITHHOLD_STAGE, -1)
        bs.fp8_debug_set(bs.FP8_DEBUG_WAIT_LIMIT_CYCLES, 0)
    compare(bs.fp8_moe_layer(x, w, ids, *layer.weights, workspace=space), *layer.reference(x, w, ids))
    assert bs.fp8_status_query() == 0


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["layer", "route"])
def test_outputs_belong_to_the_stream_that_writes_them(name, handle):
    """Memory freed on the current stream may still be in use by its queued work: a call on
    another stream must not be given it."""
    layer = _moe.Layer(4, 1024, 512, 6)
    x, w, ids = _moe.inputs(64, 2, 4, 1024, 7)
    logits = torch.randn(2048, 256, device="cuda")

    def call(stream=None):
        if name == "layer":
            return bs.fp8_moe_layer(x, w, ids, *layer.weights, stream=stream)
        return bs.fp8_moe_route(logits, 8, order=False, stream=stream)[1]
    first = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    where = first.data_ptr()
    want = first.clone()
    del first
    got = call(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert got.data_ptr() != where and torch.equal(got, want)


@pytest.mark.parametrize("H,I", [(1040, 528), (2064, 1040)])
def test_two_calls_at_once_with_workspaces_of_their_own(H, I):   # noqa: E741
    layer = _moe.Layer(8, H, I, 6)
    sets = [_moe.inputs(T, 3, 8, H, T) for T in (8, 30, 64, 17)]
    want = [bs.fp8_moe_layer(*s, *layer.weights) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [bs.fp8_moe_layer(*s, *layer.weights, stream=t) for s, t in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
