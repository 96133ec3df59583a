"""Workloads of the 128-granular FP8 operators, each in two forms.

Three operators of a served mixture-of-experts (or dense) layer: the matrix product
with one scale for each 1 x 128 piece of a token and each 128 x 128 block of a weight
(``gemm``), the same product grouped by expert over ragged, device-resident row counts
(``experts``), and the quantizer that makes their activations (``quant``: plain,
gathered by a router's row list, or of the gated activation between the two products).

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
        # one token through a projection of a decoding step: latency and the weight's bytes
        {"name": "gemm 1 token", "op": "gemm", "M": 1, "N": 4096, "K": 7168, "pow2": False},
        # a decoding batch of odd size, N and K that end inside a 128 block
        {"name": "gemm 37 tokens ragged", "op": "gemm", "M": 37, "N": 4104, "K": 7184, "pow2": False},
        # the square product of the benchmark
        {"name": "gemm 4096 square", "op": "gemm", "M": 4096, "N": 4096, "K": 4096, "pow2": False},
        # the prefill projection of the benchmark, any scales and power-of-two scales
        {"name": "gemm prefill", "op": "gemm", "M": 8192, "N": 28672, "K": 8192, "pow2": False},
        {"name": "gemm prefill pow2", "op": "gemm", "M": 8192, "N": 28672, "K": 8192, "pow2": True},
        # three tokens of eight experts each out of 64: one or two rows for an expert, most without any
        {"name": "experts 24 rows of 64", "op": "experts", "E": 64, "T": 24, "N": 4096, "K": 7168,
         "spread": "even", "route": 3, "pow2": False},
        # the benchmark's decode groups: 16 experts with 1 to 64 rows
        {"name": "experts decode", "op": "experts", "E": 16, "T": 532, "N": 4096, "K": 7168,
         "spread": "even", "route": 1, "pow2": False},
        # a short prompt over 32 experts, a few of which take most of the rows, sizes that end inside blocks
        {"name": "experts skewed ragged", "op": "experts", "E": 32, "T": 4001, "N": 4104, "K": 2064,
         "spread": "skewed", "route": 2, "pow2": False},
        # a long prompt: about a thousand rows for an expert
        {"name": "experts prefill", "op": "experts", "E": 16, "T": 16384, "N": 4096, "K": 7168,
         "spread": "even", "route": 4, "pow2": False},
        # one token's activations before a projection
        {"name": "quant 1 token", "op": "quant", "form": "plain", "M": 1, "K": 7168, "pow2": False},
        # a prompt's tokens gathered into expert order, four experts each
        {"name": "quant gathered", "op": "quant", "form": "gather", "M": 16384, "K": 7168, "pow2": True},
        # the gated activation of a prompt between the two products, an odd number of rows
        {"name": "quant swiglu", "op": "quant", "form": "swiglu", "M": 16001, "K": 4096, "pow2": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "experts", "experts", "quant"])
    pow2 = rng.random() < 0.3
    if op == "gemm":
        return {"op": op, "M": _log(rng, 1, 8192), "N": 8 * _log(rng, 8, 2048), "K": 16 * _log(rng, 8, 512),
                "pow2": pow2}
    if op == "experts":
        E, N, K = _log(rng, 2, 64), 8 * _log(rng, 16, 512), 16 * _log(rng, 8, 448)
        return {"op": op, "E": E, "T": _log(rng, 1, 16384), "N": N, "K": K,
                "spread": rng.choice(["even", "skewed"]), "route": rng.randrange(1, 1 << 20), "pow2": pow2}
    return {"op": op, "form": rng.choice(["plain", "gather", "swiglu"]), "M": _log(rng, 1, 16384),
            "K": 16 * _log(rng, 4, 448), "pow2": pow2}


def rows_of(case):
    """The row count of each expert: every row goes to an expert by the expert's weight."""
    r = random.Random(case["route"])
    E = case["E"]
    w = [1.0 if case["spread"] == "even" else math.exp(1.5 * r.gauss(0, 1)) for _ in range(E)]
    dead = [case["spread"] == "skewed" and e % 5 == 4 for e in range(E)]
    w = [0.0 if d else v for v, d in zip(w, dead)]
    picks = r.choices(range(E), weights=w, k=case["T"])
    return [picks.count(e) for e in range(E)]


def work(case):
    K = case["K"]
    if case["op"] == "quant":
        M = case["M"]
        x = M * K * (4 if case["form"] == "swiglu" else 2)
        if case["form"] == "gather":   # each token is read once, and the row list
            x = tokens_of(case) * K * 2 + 4 * M
        return {"bytes": x + M * K + 4 * M * blocks(K), "flops": M * K * (12 if case["form"] == "swiglu" else 3)}
    N = case["N"]
    b = N * K + 4 * blocks(N) * blocks(K)
    if case["op"] == "gemm":
        M, n = case["M"], 1
    else:
        rows = rows_of(case)
        M, n = case["T"], sum(m > 0 for m in rows)
    return {"bytes": n * b + M * K + 4 * M * blocks(K) + 2 * M * N, "flops": 2 * M * N * K}


def tokens_of(case):
    return max(1, case["M"] // 4)


# ------------------------------------------------------------------ inputs ----

def _scale(amax, pow2):
    # divided by a tensor: by a Python number, torch multiplies by the rounded reciprocal
    s = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    if pow2:
        s = ((s.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32)   # up to a power of two
    return s


def _quantized(x, rows, pow2):
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


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 11)
    K, pow2 = case["K"], bool(case["pow2"])
    st = dict(case)
    if case["op"] == "quant":
        M = case["M"]
        if case["form"] == "gather":
            n = tokens_of(case)
            st["x"] = _activations(n, K, g, dev)
            st["rows"] = torch.randperm(4 * n + 4, generator=g, device=dev)[:M].remainder(n).to(torch.int32)
        elif case["form"] == "swiglu":
            st["x"] = (torch.randn(M, 2 * K, generator=g, device=dev) * 2).to(torch.bfloat16)
        else:
            st["x"] = _activations(M, K, g, dev)
        st["q"] = torch.empty(M, K, dtype=torch.uint8, device=dev)
        st["s"] = torch.empty(M, blocks(K), dtype=torch.float32, device=dev)
        return st
    N = case["N"]
    if case["op"] == "gemm":
        M = case["M"]
        st["B"], st["sB"] = _quantized(torch.randn(N, K, generator=g, device=dev) * 0.02, G, pow2)
    else:
        M, E = case["T"], case["E"]
        rows = rows_of(case)
        st["B"] = torch.empty(E, N, K, dtype=torch.uint8, device=dev)
        st["sB"] = torch.empty(E, blocks(N), blocks(K), dtype=torch.float32, device=dev)
        for e in range(E):
            st["B"][e], st["sB"][e] = _quantized(torch.randn(N, K, generator=g, device=dev) * 0.02, G, pow2)
        ends = [sum(rows[:e + 1]) for e in range(E)]
        st["offsets"] = torch.tensor([0] + ends, dtype=torch.int32, device=dev)
        st["busy"] = torch.tensor([e for e in range(E) if rows[e]], dtype=torch.int64, device=dev)
        st["most"] = max(rows)
    st["A"], st["sA"] = _quantized(_activations(M, K, g, dev), 1, pow2)
    st["C"] = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    return st


# -------------------------------------------------------------- plain forms ----

def _values(q, s, rows):
    """fp32 values of codes [..., R, K] with a scale per `rows` x 128 block."""
    R, K = q.shape[-2:]
    full = s.repeat_interleave(rows, -2)[..., :R, :].repeat_interleave(G, -1)[..., :K]
    return q.view(F8).float() * full


def plain_gemm(st):
    a, b = _values(st["A"], st["sA"], 1), _values(st["B"], st["sB"], G)
    return (a @ b.T).to(torch.bfloat16)


def plain_experts(st):
    """The rows of each expert that has any, padded to the longest, in one batched product."""
    off, busy = st["offsets"].long(), st["busy"]
    row = torch.arange(st["T"], device=off.device)
    start, end = off[busy], off[busy + 1]
    e = torch.searchsorted(end, row, right=True)
    slot = row - start[e]
    a = torch.zeros(busy.shape[0], st["most"], st["K"], device=off.device)
    a[e, slot] = _values(st["A"], st["sA"], 1)
    b = _values(st["B"][busy], st["sB"][busy], G)
    return torch.bmm(a, b.transpose(1, 2))[e, slot].to(torch.bfloat16)


def plain_quant(st):
    x, K = st["x"], st["K"]
    if st["form"] == "gather":
        x = x[st["rows"].long()]
    x = x.float()
    if st["form"] == "swiglu":
        gate, up = x[:, :K], x[:, K:]
        x = gate / (1 + torch.exp(-gate)) * up
    p = torch.nn.functional.pad(x, (0, blocks(K) * G - K)).view(x.shape[0], blocks(K), G)
    s = _scale(p.abs().amax(dim=2), st["pow2"])
    q = (p / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8)
    return {"q": q.view(x.shape[0], -1)[:, :K].contiguous(), "s": s}


# --------------------------------------------------------------------- run ----

def run(state):
    if not own:
        return {"gemm": plain_gemm, "experts": plain_experts, "quant": plain_quant}[state["op"]](state)
    import block_scaled_fp8_sm_gb300 as bs
    mode = bs.FP8_PATH_NATIVE if state["pow2"] else None
    if state["op"] == "gemm":
        return bs.fp8_gemm_block128(state["A"], state["sA"], state["B"], state["sB"], state["C"], mode=mode)
    if state["op"] == "experts":
        return bs.fp8_gemm_experts(state["A"], state["sA"], state["B"], state["sB"], state["C"], state["offsets"],
                                   mode=mode)
    if state["form"] == "swiglu":
        q, s = bs.fp8_swiglu_quantize_tokens(state["x"], state["q"], state["s"], pow2=state["pow2"])
    else:
        q, s = bs.fp8_quantize_tokens(state["x"], state["q"], state["s"], rows=state.get("rows"), pow2=state["pow2"])
    return {"q": q.view(F8), "s": s}


# ----------------------------------------------------- the definition, 64 bits ----

def _e4m3_table(dev):
    """The 256 values of E4M3 by its definition: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(float("nan") if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _power(v, up):
    """The power of two at or next to positive v, by the bits of a double (logarithms and ldexp may miss it)."""
    low = (1 << 52) - 1
    return ((v.contiguous().view(torch.int64) + (low if up else 0)) & ~low).view(torch.float64)


def _exact_product(A, sA, B, sB):
    t = _e4m3_table(A.device)
    K = A.shape[1]
    out = torch.zeros(A.shape[0], B.shape[0], dtype=torch.float64, device=A.device)
    for k in range(0, K, G * 16):   # sixteen blocks of K at a time: the values fit beside the operands
        part = slice(k, min(K, k + G * 16))
        at = torch.arange(part.start, part.stop, device=A.device) // G
        a = t[A[:, part].int()] * sA.double()[:, at]
        b = t[B[:, part].int()] * sB.double()[torch.arange(B.shape[0], device=A.device) // G][:, at]
        out += a @ b.T
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gemm":
        return _exact_product(st["A"], st["sA"], st["B"], st["sB"])
    if case["op"] == "experts":
        ends = st["offsets"].tolist()
        return torch.cat([_exact_product(st["A"][a:b], st["sA"][a:b], st["B"][e], st["sB"][e])
                          for e, (a, b) in enumerate(zip(ends, ends[1:])) if b > a])
    x = st["x"].double()
    K = case["K"]
    if case["form"] == "gather":
        x = x.index_select(0, st["rows"].long())
    if case["form"] == "swiglu":
        x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
    q, s = torch.empty_like(x), torch.empty(x.shape[0], blocks(K), dtype=torch.float64, device=x.device)
    for b in range(blocks(K)):
        v = x[:, b * G:(b + 1) * G]
        top = v.abs().amax(dim=1)
        one = torch.where(top > 0, top / torch.full_like(top, E4M3_MAX), torch.ones_like(top))
        if case["pow2"]:
            one = _power(one, up=True)
        v = v / one[:, None]
        step = _power(v.abs().clamp(min=2.0 ** -6), up=False) / 8
        q[:, b * G:(b + 1) * G] = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        s[:, b] = one
    return {"q": q, "s": s}
