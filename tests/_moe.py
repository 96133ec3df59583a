"""Inputs and 64-bit references of the router and of the mixture-of-experts layer (torch, no
library code)."""
import math

import torch

from tests._fused import values


def route(logits, top, sigmoid=False, renormalize=True, scale=1.0):
    """(weights, ids, offsets, rows, places, tolerance of the weights), in 64 bits."""
    v = logits.double()
    T, E = v.shape
    v = torch.where(v.isnan(), torch.full_like(v, -math.inf), v)
    left, ids = v.clone(), torch.full((T, top), -1, dtype=torch.int64)
    at = torch.arange(E).expand(T, E)
    for j in range(top):
        best = left.amax(1, keepdim=True) if E else left
        i = torch.where(left == best, at, torch.full_like(at, E)).amin(1, keepdim=True)
        ids[:, j:j + 1] = torch.where(best == -math.inf, torch.full_like(i, -1), i)
        left.scatter_(1, i, -math.inf)
    val = torch.where(ids >= 0, v.gather(1, ids.clamp(min=0)), torch.full((T, top), -math.inf, dtype=torch.float64))
    m = torch.where(val[:, :1] == -math.inf, torch.zeros_like(val[:, :1]), val[:, :1])

    def below(x):   # exp(x - m); the largest gives 1 even where it is infinite
        return torch.where(x == m, torch.ones_like(x), torch.exp(x - m))
    p = torch.sigmoid(val) if sigmoid else below(val)
    if sigmoid and renormalize:   # common factor exp(-m) where all are small
        f = m.clamp(max=0)
        p = torch.where(val > 0, p, torch.exp(val - f) / (1 + torch.exp(val.clamp(max=0))))
    p = torch.where(ids >= 0, p, torch.zeros_like(p))
    if renormalize:
        total = p.sum(1, keepdim=True)
    else:
        total = torch.ones_like(m) if sigmoid else torch.where(v == -math.inf, torch.zeros_like(v), below(v)).sum(1, keepdim=True)
    w = torch.where(ids >= 0, p / total, torch.zeros_like(p)) * scale
    # fp32: the argument of exp is rounded by 2^-24 |v - m|; exp, the sum's at most ten
    # additions in a row, the division and the scale by a few steps of 2^-24 each
    reach = torch.where(ids >= 0, (val - m).abs().nan_to_num(0, 0, 0) + val.abs().nan_to_num(0, 0, 0), torch.zeros_like(p))
    tol = w.abs() * (2 * reach + 32) * 2.0 ** -24 + 2.0 ** -140
    flat = ids.flatten()
    offsets, rows, places = [0], torch.full_like(flat, -1), torch.full_like(flat, -1)
    for e in range(E):
        mine = torch.nonzero(flat == e).flatten()
        a, b = offsets[-1], offsets[-1] + mine.numel()
        offsets.append(b)
        rows[a:b] = mine // top
        places[mine] = torch.arange(a, b)
    return w, ids, torch.tensor(offsets), rows, places.view(T, top), tol


class Layer:
    """Weights of a layer on the GPU: codes and 128 x 128 scales."""

    def __init__(self, E, H, I, seed):   # noqa: E741
        g = torch.Generator().manual_seed(seed)
        self.E, self.H, self.I = E, H, I

        def weight(N, K):
            q = torch.randn(E * N, K, generator=g).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s = (torch.rand(E, -(-N // 128), -(-K // 128), generator=g) + 0.5) * K ** -0.5
            return q.view(E, N, K).cuda(), s.cuda()
        self.gate_up, self.s_gate_up = weight(2 * I, H)
        self.down, self.s_down = weight(H, I)

    @property
    def weights(self):
        return self.gate_up, self.s_gate_up, self.down, self.s_down

    def reference(self, x, w, ids):
        """(out, bound) in 64 bits.  The sums of a product are off by at most 1e-5 of their
        magnitude (the products' own bound; fp16 holds x and the codes exactly); silu has
        slopes up to 1.1 and is off by 2^-14 of itself; h is rounded by 2^-11 (fp16); the
        result by 2^-8 (bf16)."""
        out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        near = torch.zeros_like(out)
        xd, top = x.double(), ids.shape[1]
        flat = ids.flatten().tolist()
        for e in sorted({v for v in flat if 0 <= v < self.E}):
            pairs = torch.tensor([p for p, v in enumerate(flat) if v == e], device=x.device)
            token, f = pairs // top, w.flatten()[pairs].double()[:, None]
            W, D = values(self.gate_up[e], self.s_gate_up[e], 128), values(self.down[e], self.s_down[e], 128)
            gate, up = (xd[token] @ W.T).split(self.I, 1)
            tg, tu = (xd[token].abs() @ W.abs().T).split(self.I, 1)
            s = gate * torch.sigmoid(gate)
            h = s * up
            dh = (2.0 ** -11 + 2.0 ** -13) * h.abs() + 1e-5 * (1.1 * tg * up.abs() + s.abs() * tu)
            out.index_add_(0, token, f * (h @ D.T))
            near.index_add_(0, token, f.abs() * ((dh + 1e-5 * h.abs()) @ D.abs().T))
        return out, near + 2.0 ** -8 * out.abs() + 2.0 ** -134


def inputs(T, top, E, H, seed):
    """x [T, H], weights and ids [T, top] (distinct experts of a token) on the GPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g)
    x = torch.where(torch.rand(T, H, generator=g) < 0.01, x * 40, x).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(T)]).to(torch.int32)
    w = torch.rand(T, top, generator=g) + 0.05
    return x.cuda(), (w / w.sum(1, keepdim=True)).cuda(), ids.cuda()
