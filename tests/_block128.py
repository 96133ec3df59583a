"""Inputs and 64-bit references of the 128-granular operators' tests (numpy and
torch on the CPU; no library code)."""
import numpy as np
import torch

G = 128


def blocks(n):
    return -(-n // G)


def e4m3_table():
    """The 256 values of E4M3 from its definition (1 sign, 4 exponent, 3 mantissa
    bits, bias 7; the two all-ones codes are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 128, -v, v)
    v[(c & 127) == 127] = np.nan
    return v


TABLE = e4m3_table()


def codes(rows, K, g, scale=1.0):
    x = torch.randn(rows, K, generator=g) * scale
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def scales(shape, g, pow2):
    if pow2:
        return torch.ldexp(torch.ones(shape), torch.randint(-6, 4, shape, generator=g)).float()
    return (torch.rand(shape, generator=g) * 2 + 0.05).float()


class Product:
    """C = A B^T with scales; lead = () for one product or (E,) for experts."""

    def __init__(self, M, N, K, seed, pow2=False, E=None):
        g = torch.Generator().manual_seed(seed)
        self.M, self.N, self.K, self.E = M, N, K, E
        self.A = codes(M, K, g, 2.0)
        self.sA = scales((M, blocks(K)), g, pow2)
        n = 1 if E is None else E
        self.B = codes(n * N, K, g).view(n, N, K)
        self.sB = scales((n, blocks(N), blocks(K)), g, pow2)
        if E is None:
            self.B, self.sB = self.B[0], self.sB[0]

    def on(self, dev):
        return [t.to(dev) for t in (self.A, self.sA, self.B, self.sB)]


def values(q, s, rows):
    """float64 values of codes q [R, K] with a scale per `rows` x 128 block."""
    R, K = q.shape
    full = np.repeat(np.repeat(s.numpy().astype(np.float64), rows, 0)[:R], G, 1)[:, :K]
    return TABLE[q.numpy()] * full


def product(A, sA, B, sB):
    """(C, T) in float64: the result and its magnitude sum."""
    a, b = values(A, sA, 1), values(B, sB, G)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def quantized(y, pow2=False):
    """(codes' values, scales) in float64 of y [M, K] float64: s from the correctly
    rounded fp32 quotient max|y| / 448, then the nearest E4M3 value of the fp32 quotient
    y / s, ties to the even code, saturating."""
    M, K = y.shape
    q, s = np.zeros_like(y), np.zeros((M, blocks(K)))
    for b in range(blocks(K)):
        v = y[:, b * G:(b + 1) * G]
        top = np.abs(v).max(axis=1)
        one = np.where(top > 0, (top / 448.0).astype(np.float32).astype(np.float64), 1.0)
        if pow2:
            m, e = np.frexp(one)
            one = np.maximum(np.ldexp(1.0, np.where(m > 0.5, e, e - 1)), 2.0 ** -126)
        v = (v / one[:, None]).astype(np.float32).astype(np.float64)
        _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
        step = np.ldexp(1.0, e - 4)
        q[:, b * G:(b + 1) * G] = np.clip(np.rint(v / step) * step, -448, 448)
        s[:, b] = one
    return q, s
