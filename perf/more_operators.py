"""Workloads of the operators around the 128-granular FP8 products, each in two forms.

Three operators of a served dense or mixture-of-experts layer: the matrix product with
bias, activation and residual in its epilogue (``fused``), the whole mixture-of-experts
layer of a few tokens, from bf16 activations to the weighted sum of their experts
(``moe``), and the router that picks each token's experts and puts the rows in expert
order (``route``).

``own`` False computes an operator in plain fp32 torch arithmetic, rounded once at the
end; ``own`` True calls the library.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
G = 128
F8 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // G)


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # one token through a projection with a bias and an activation: latency and the weight's bytes
        {"name": "fused 1 token", "op": "fused", "M": 1, "N": 4096, "K": 7168, "act": "silu", "bias": "f32",
         "residual": False, "pow2": False},
        # a decoding batch of odd size through an output projection onto its residual, ends inside 128 blocks
        {"name": "fused 37 tokens ragged", "op": "fused", "M": 37, "N": 4104, "K": 7184, "act": "gelu",
         "bias": "bf16", "residual": True, "pow2": False},
        # the square product of the benchmark with every part of the epilogue
        {"name": "fused 4096 square", "op": "fused", "M": 4096, "N": 4096, "K": 4096, "act": "gelu_tanh",
         "bias": "bf16", "residual": True, "pow2": False},
        # the prefill projection of the benchmark, power-of-two scales, bias and activation
        {"name": "fused prefill pow2", "op": "fused", "M": 8192, "N": 28672, "K": 8192, "act": "gelu",
         "bias": "f32", "residual": False, "pow2": True},
        # one token through the example's layer: latency
        {"name": "moe 1 token", "op": "moe", "T": 1, "top": 4, "E": 32, "H": 2048, "I": 1024, "route": 5,
         "padded": 0},
        # three tokens of eight experts each out of 64: one or two rows for an expert, the weights' bytes
        {"name": "moe 3 tokens", "op": "moe", "T": 3, "top": 8, "E": 64, "H": 7168, "I": 2048, "route": 3,
         "padded": 0},
        # a decoding batch padded to a captured size, sizes that end inside 128 blocks
        {"name": "moe 19 tokens ragged", "op": "moe", "T": 19, "top": 3, "E": 16, "H": 2064, "I": 1040, "route": 7,
         "padded": 3},
        # the largest batch that the layer takes: every expert is busy, eight rows each on average
        {"name": "moe 64 tokens", "op": "moe", "T": 64, "top": 8, "E": 64, "H": 7168, "I": 2048, "route": 9,
         "padded": 0},
        # one token's router in a decoding step: latency
        {"name": "route 1 token", "op": "route", "T": 1, "E": 64, "top": 8, "type": "f32", "sigmoid": False,
         "masked": False},
        # a decoding batch, half-precision logits (with ties), experts and padding rows masked
        {"name": "route 37 tokens masked", "op": "route", "T": 37, "E": 96, "top": 6, "type": "bf16",
         "sigmoid": True, "masked": True},
        # a prompt over 64 experts
        {"name": "route prompt", "op": "route", "T": 16384, "E": 64, "top": 4, "type": "f32", "sigmoid": False,
         "masked": False},
        # a prompt of odd length over 256 experts, eight each, half of the experts closed to a token
        {"name": "route prompt masked", "op": "route", "T": 16001, "E": 256, "top": 8, "type": "f32",
         "sigmoid": True, "masked": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fused", "moe", "route"])
    if op == "fused":
        return {"op": op, "M": _log(rng, 1, 8192), "N": 8 * _log(rng, 8, 2048), "K": 16 * _log(rng, 8, 512),
                "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                "bias": rng.choice(["none", "f32", "bf16"]), "residual": rng.random() < 0.5,
                "pow2": rng.random() < 0.3}
    if op == "moe":
        E = _log(rng, 2, 64)
        return {"op": op, "T": _log(rng, 1, 64), "top": rng.randint(1, min(8, E)), "E": E,
                "H": 16 * _log(rng, 16, 448), "I": 16 * _log(rng, 8, 128), "route": rng.randrange(1, 1 << 20),
                "padded": rng.choice([0, 0, 0, 1])}
    E = _log(rng, 4, 256)
    return {"op": op, "T": _log(rng, 1, 16384), "E": E, "top": rng.randint(1, min(8, E)),
            "type": rng.choice(["f32", "bf16"]), "sigmoid": rng.random() < 0.5, "masked": rng.random() < 0.4}


def experts_of(case):
    """Each token's experts (distinct; -1 in the rows of padding)."""
    r = random.Random(case["route"])
    T = case["T"]
    live = max(1, T - case["padded"])
    return [r.sample(range(case["E"]), case["top"]) if t < live else [-1] * case["top"] for t in range(T)]


def work(case):
    if case["op"] == "route":
        T, E, top = case["T"], case["E"], case["top"]
        return {"bytes": T * E * (4 if case["type"] == "f32" else 2) + 16 * T * top + 4 * (E + 1), "flops": 4 * T * E}
    if case["op"] == "moe":
        T, H, I, ids = case["T"], case["H"], case["I"], experts_of(case)
        pairs = [e for row in ids for e in row if e >= 0]
        each = 3 * I * H + 4 * blocks(2 * I) * blocks(H) + 4 * blocks(H) * blocks(I)
        return {"bytes": len(set(pairs)) * each + 4 * T * H + 8 * T * case["top"], "flops": 6 * len(pairs) * I * H}
    M, N, K = case["M"], case["N"], case["K"]
    b = M * K + 4 * M * blocks(K) + N * K + 4 * blocks(N) * blocks(K) + 2 * M * N * (2 if case["residual"] else 1)
    return {"bytes": b + N * {"none": 0, "f32": 4, "bf16": 2}[case["bias"]], "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs ----

def _scale(amax, pow2):
    # divided by a tensor: by a Python number, torch multiplies by the rounded reciprocal
    s = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    if pow2:
        s = ((s.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32)   # up to a power of two
    return s


def _quantized(x, rows, pow2=False):
    """Codes (uint8) and scales of x [R, K], one scale per `rows` x 128 block."""
    R, K = x.shape
    p = torch.zeros(-(-R // rows) * rows, blocks(K) * G, dtype=torch.float32, device=x.device)
    p[:R, :K] = x
    p = p.view(-1, rows, blocks(K), G)
    s = _scale(p.abs().amax(dim=(1, 3)), pow2)
    q = (p / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8).view(torch.uint8)
    return q.view(-1, blocks(K) * G)[:R, :K].contiguous(), s.contiguous()


def _activations(M, K, g, dev):
    """bf16 N(0, 1) with a few outliers, as activations have."""
    x = torch.randn(M, K, generator=g, device=dev)
    return torch.where(torch.rand(M, K, generator=g, device=dev) < 0.005, x * 50, x).to(torch.bfloat16)


def _expert_weights(E, N, K, g, dev):
    q = torch.empty(E, N, K, dtype=torch.uint8, device=dev)
    s = torch.empty(E, blocks(N), blocks(K), dtype=torch.float32, device=dev)
    for e in range(E):
        q[e], s[e] = _quantized(torch.randn(N, K, generator=g, device=dev) * K ** -0.5, G)
    return q, s


def _workspace(size, *args):
    """The memory that a program keeps for the library's call (the plain forms need none)."""
    if not own:
        return None
    import block_scaled_fp8_sm_gb300 as bs
    return torch.empty(getattr(bs, size)(*args), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 6367 + 29)
    st = dict(case)
    if case["op"] == "route":
        T, E, top = case["T"], case["E"], case["top"]
        x = torch.randn(T, E, generator=g, device=dev) * 2
        if case["masked"]:
            # half of the experts are closed to a token, and some rows are padding
            shut = torch.rand(T, E, generator=g, device=dev) < 0.5
            shut |= torch.rand(T, 1, generator=g, device=dev) < 0.03
            x = torch.where(shut, torch.full_like(x, -math.inf), x)
        st["logits"] = x if case["type"] == "f32" else x.to(torch.bfloat16)
        i32 = lambda *n: torch.empty(*n, dtype=torch.int32, device=dev)   # noqa: E731
        st["out"] = (torch.empty(T, top, dtype=torch.float32, device=dev), i32(T, top), i32(E + 1), i32(T * top),
                     i32(T, top))
        st["workspace"] = _workspace("fp8_moe_route_workspace_bytes", T, E, top)
        return st
    if case["op"] == "moe":
        T, top, E, H, I = (case[k] for k in ("T", "top", "E", "H", "I"))
        st["gate_up"], st["s_gate_up"] = _expert_weights(E, 2 * I, H, g, dev)
        st["down"], st["s_down"] = _expert_weights(E, H, I, g, dev)
        st["x"] = _activations(T, H, g, dev)
        ids = experts_of(case)
        st["ids"] = torch.tensor(ids, dtype=torch.int32, device=dev)
        st["busy"] = sorted({e for row in ids for e in row if e >= 0})
        w = torch.rand(T, top, generator=g, device=dev) + 0.05
        st["weights"] = torch.where(st["ids"] >= 0, w / w.sum(1, keepdim=True), torch.zeros_like(w))
        st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        st["workspace"] = _workspace("fp8_moe_layer_workspace_bytes", T, top, I)
        return st
    M, N, K, pow2 = case["M"], case["N"], case["K"], bool(case["pow2"])
    st["B"], st["sB"] = _quantized(torch.randn(N, K, generator=g, device=dev) * K ** -0.5, G, pow2)
    st["A"], st["sA"] = _quantized(_activations(M, K, g, dev), 1, pow2)
    bias = torch.randn(N, generator=g, device=dev) * 0.5
    st["b"] = {"none": None, "f32": bias, "bf16": bias.to(torch.bfloat16)}[case["bias"]]
    st["R"] = torch.randn(M, N, generator=g, device=dev).to(torch.bfloat16) if case["residual"] else None
    st["C"] = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    return st


# -------------------------------------------------------------- plain forms ----

def _values(q, s, rows):
    """fp32 values of codes [R, K] with a scale per `rows` x 128 block."""
    R, K = q.shape
    full = s.repeat_interleave(rows, 0)[:R].repeat_interleave(G, 1)[:, :K]
    return q.view(F8).float() * full


def _activated(y, act):
    if act == "relu":
        return torch.relu(y)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":   # y Phi(y); erfc keeps the tail
        return 0.5 * y * torch.erfc(y * -math.sqrt(0.5))
    if act == "gelu_tanh":   # 0.5 y (1 + tanh u) = y / (1 + exp(-2 u))
        return y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def plain_fused(st):
    y = _values(st["A"], st["sA"], 1) @ _values(st["B"], st["sB"], G).T
    if st["b"] is not None:
        y = y + st["b"].float()
    y = _activated(y, st["act"])
    if st["R"] is not None:
        y = y + st["R"].float()
    return y.to(torch.bfloat16)


def plain_moe(st):
    x, I = st["x"].float(), st["I"]
    out = torch.zeros_like(x)
    for e in st["busy"]:
        gu = x @ _values(st["gate_up"][e], st["s_gate_up"][e], G).T
        h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
        w = (st["weights"] * (st["ids"] == e)).sum(1, keepdim=True)   # 0 for tokens that are not this expert's
        out += w * (h @ _values(st["down"][e], st["s_down"][e], G).T)
    return out.to(torch.bfloat16)


def plain_route(st):
    x, E, top = st["logits"].float(), st["E"], st["top"]
    T = x.shape[0]
    v, ids = torch.sort(x, dim=1, descending=True, stable=True)   # equal logits: the lower expert first
    v, ids = v[:, :top], ids[:, :top]
    none = v == -math.inf
    m = v[:, :1]
    if st["sigmoid"]:   # sigmoid(v) / sum, scaled by exp(-m), m the largest logit where that is below 0
        m = torch.where(none[:, :1], torch.zeros_like(m), m).clamp(max=0)
        p = torch.exp(v - m) / (1 + torch.exp(v))
        p = torch.where(v > 0, 1 / (1 + torch.exp(-v)), p)
    else:
        p = torch.exp(v - m)
    p = torch.where(none, torch.zeros_like(p), p)
    s = p.sum(1, keepdim=True)
    weights = torch.where(none, torch.zeros_like(p), p / s)
    key = torch.where(none, torch.full_like(ids, E), ids).flatten()
    count = torch.zeros(E + 1, dtype=torch.int64, device=x.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([count[:1] * 0, torch.cumsum(count[:E], 0)])
    order = torch.sort(key, stable=True).indices   # pairs in expert order
    place = torch.empty_like(order)
    place[order] = torch.arange(T * top, device=x.device)
    gone = none.flatten()
    rows = torch.where(gone[order], torch.full_like(order, -1), order // top)
    place = torch.where(gone, torch.full_like(place, -1), place).view(T, top)
    i32 = lambda t: t.to(torch.int32)   # noqa: E731
    return {"weights": weights, "ids": i32(torch.where(none, torch.full_like(ids, -1), ids)), "offsets": i32(offsets),
            "rows": i32(rows), "places": i32(place)}


# --------------------------------------------------------------------- run ----

def run(state):
    if not own:
        return {"fused": plain_fused, "moe": plain_moe, "route": plain_route}[state["op"]](state)
    import block_scaled_fp8_sm_gb300 as bs
    if state["op"] == "fused":
        act = {"none": bs.FP8_ACT_NONE, "relu": bs.FP8_ACT_RELU, "gelu": bs.FP8_ACT_GELU,
               "gelu_tanh": bs.FP8_ACT_GELU_TANH, "silu": bs.FP8_ACT_SILU}[state["act"]]
        return bs.fp8_gemm_block128_fused(state["A"], state["sA"], state["B"], state["sB"], state["C"],
                                          bias=state["b"], act=act, residual=state["R"],
                                          mode=bs.FP8_PATH_NATIVE if state["pow2"] else None)
    if state["op"] == "moe":
        return bs.fp8_moe_layer(state["x"], state["weights"], state["ids"], state["gate_up"], state["s_gate_up"],
                                state["down"], state["s_down"], state["out"], state["workspace"])
    weights, ids, offsets, rows, places = bs.fp8_moe_route(state["logits"], state["top"], sigmoid=state["sigmoid"],
                                                           out=state["out"], workspace=state["workspace"])
    return {"weights": weights, "ids": ids, "offsets": offsets, "rows": rows, "places": places}


# ----------------------------------------------------- the definition, 64 bits ----

def _e4m3_table(dev):
    """The 256 values of E4M3 by its definition: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(float("nan") if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _weight(q, s, table):
    """Codes [N, K] and their 128 x 128 scales in 64 bits."""
    n = torch.arange(q.shape[0], device=q.device) // G
    k = torch.arange(q.shape[1], device=q.device) // G
    return table[q.int()] * s.double()[n][:, k]


def _exact_fused(st):
    t = _e4m3_table(st["A"].device)
    M, K = st["A"].shape
    N = st["B"].shape[0]
    y = torch.zeros(M, N, dtype=torch.float64, device=t.device)
    for k in range(0, K, G * 16):   # sixteen blocks of K at a time: the values fit beside the operands
        part = slice(k, min(K, k + G * 16))
        at = slice(k // G, blocks(part.stop))
        a = t[st["A"][:, part].int()] * st["sA"].double()[:, at].repeat_interleave(G, 1)[:, :part.stop - k]
        y += a @ _weight(st["B"][:, part], st["sB"][:, at], t).T
    if st["b"] is not None:
        y += st["b"].double()
    if st["act"] == "relu":
        y.clamp_(min=0)
    elif st["act"] == "silu":
        y *= torch.sigmoid(y)
    elif st["act"] == "gelu":
        y *= torch.special.erfc(y / -math.sqrt(2)) / 2
    elif st["act"] == "gelu_tanh":
        y *= torch.sigmoid((y + 0.044715 * y ** 3) * math.sqrt(8 / math.pi))
    return y if st["R"] is None else y + st["R"].double()


def _exact_moe(st):
    t = _e4m3_table(st["x"].device)
    x, I, top = st["x"].double(), st["I"], st["top"]
    out = torch.zeros_like(x)
    flat = st["ids"].flatten().tolist()
    for e in sorted(set(flat) - {-1}):
        pairs = torch.tensor([p for p, v in enumerate(flat) if v == e], device=x.device)
        token = pairs // top
        gate, up = (x[token] @ _weight(st["gate_up"][e], st["s_gate_up"][e], t).T).split(I, dim=1)
        y = (gate * torch.sigmoid(gate) * up) @ _weight(st["down"][e], st["s_down"][e], t).T
        out.index_add_(0, token, y * st["weights"].flatten()[pairs].double()[:, None])
    return out


def _exact_route(st):
    v, E, top = st["logits"].double(), st["E"], st["top"]
    T = v.shape[0]
    at = torch.arange(E, device=v.device).expand(T, E)
    left, picks, values = v.clone(), [], []
    for _ in range(top):   # the largest that is left, the lowest expert of equal ones
        best = left.amax(dim=1, keepdim=True)
        i = torch.where(left == best, at, torch.full_like(at, E)).amin(dim=1, keepdim=True)
        picks.append(torch.where(best == -math.inf, torch.full_like(i, -1), i))
        values.append(best)
        left.scatter_(1, i, -math.inf)
    ids, val = torch.cat(picks, 1), torch.cat(values, 1)
    score = torch.sigmoid(val) if st["sigmoid"] else torch.exp(val - val.clamp(min=-1e300).amax(1, keepdim=True))
    score = torch.where(ids >= 0, score, torch.zeros_like(score))
    weights = score / score.sum(1, keepdim=True).clamp(min=1e-300)
    flat = ids.flatten()
    offsets, rows = [0], torch.full_like(flat, -1)
    places = torch.full_like(flat, -1)
    for e in range(E):
        mine = torch.nonzero(flat == e).flatten()
        at0 = offsets[-1]
        offsets.append(at0 + mine.numel())
        rows[at0:offsets[-1]] = torch.div(mine, top, rounding_mode="floor")
        places[mine] = torch.arange(at0, offsets[-1], device=v.device)
    return {"weights": weights, "ids": ids.int(), "offsets": torch.tensor(offsets, dtype=torch.int32, device=v.device),
            "rows": rows.int(), "places": places.view(T, top).int()}


def exact(case, seed):
    return {"fused": _exact_fused, "moe": _exact_moe, "route": _exact_route}[case["op"]](prepare(case, seed))
