"""64-bit references of the fused epilogue and the mixture-of-experts operators (torch,
no library code)."""
import math

import torch

from tests._block128 import G, TABLE

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def values(q, s, rows):
    """float64 values of codes q [R, K] (uint8) with a scale per `rows` x 128 block."""
    R, K = q.shape
    table = torch.tensor(TABLE, dtype=torch.float64, device=q.device)
    return table[q.int()] * s.double().repeat_interleave(rows, 0)[:R].repeat_interleave(G, 1)[:, :K]


def activation(y, act):
    if act == "relu":
        return torch.where(y < 0, torch.zeros_like(y), y)
    if act == "gelu":
        return y * torch.special.erfc(y * -math.sqrt(0.5)) / 2
    if act == "gelu_tanh":
        return y * torch.sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3))
    if act == "silu":
        return y * torch.sigmoid(y)
    return y


def fused(A, sA, B, sB, bias, act, R):
    """(C, bound): the result, and how far an fp32 evaluation rounded once to bf16 may be
    from it.  The sum is off by at most 1e-5 of its magnitude sum (the products' own bound),
    which an activation stretches by at most 1.13 (the largest slope of all of them); the
    activation's own error is below 2^-14 of it, adding the residual rounds by 2^-24 of each
    part, and the rounding to bf16 by 2^-8 of the result (2^-134 where it is subnormal)."""
    a, b = values(A, sA, 1), values(B, sB, G)
    y, T = a @ b.T, a.abs() @ b.abs().T
    if bias is not None:
        y, T = y + bias.double(), T + bias.double().abs()
    f = activation(y, act)
    C = f if R is None else f + R.double()
    bound = 1.13e-5 * T + 2.0 ** -14 * f.abs() + 2.0 ** -8 * C.abs() + 2.0 ** -134
    return C, bound if R is None else bound + 2.0 ** -23 * R.double().abs()
