"""A mixture-of-experts layer served in FP8: the 128-granular operators together.

    python examples/moe_layer.py [--tokens 512] [--experts 32] [--top 4] [--hidden 2048] [--inner 1024]

A router picks ``top`` experts for each token and puts the rows in expert order.  Up to
FP8_MOE_MAX_TOKENS tokens (a decoding step) go through the whole layer in one call, on
unquantized activations.  More tokens' activations are quantized in expert order (a gather
and a quantization in one pass), multiplied by each expert's gate and up weights, gated and
quantized again, multiplied by its down weights, and summed per token with the router's
weights.  The layer keeps its weights as E4M3 codes with 128 x 128 scales.  The result is
compared with the same layer in fp32 on the same (dequantized) weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_sm_gb300 as bs  # noqa: E402

BLOCK = 128


def pack_weight(w):
    """E4M3 codes and 128 x 128 fp32 scales of w [E, N, K] (once, when the model is loaded)."""
    E, N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    p = torch.zeros(E, nb * BLOCK, kb * BLOCK, device=w.device)
    p[:, :N, :K] = w
    p = p.view(E, nb, BLOCK, kb, BLOCK)
    s = p.abs().amax(dim=(2, 4)) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (p / s[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).view(E, nb * BLOCK, kb * BLOCK)[:, :N, :K].contiguous()
    return q, s.contiguous()


def unpack_weight(q, s):
    full = s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]].repeat_interleave(BLOCK, 2)[:, :, :q.shape[2]]
    return q.view(torch.float8_e4m3fn).float() * full


class MoeLayer:
    """Weights and router of one layer; ``forward`` enqueues the whole layer on the current
    stream and reads nothing back, so it can be captured in a CUDA graph."""

    def __init__(self, hidden, inner, experts, top, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.top, self.experts = top, experts
        self.router = torch.randn(experts, hidden, generator=g, device=device) * hidden ** -0.5
        self.gate_up = pack_weight(torch.randn(experts, 2 * inner, hidden, generator=g, device=device) * hidden ** -0.5)
        self.down = pack_weight(torch.randn(experts, hidden, inner, generator=g, device=device) * inner ** -0.5)

    def route(self, x):
        """(weights [T, top], ids [T, top], offsets [E + 1], token of each row in expert
        order, places [T, top] of the tokens' rows there)."""
        return bs.fp8_moe_route(x.float() @ self.router.T, self.top)

    def forward(self, x):
        T, hidden = x.shape
        w, ids, offsets, token, places = self.route(x)
        if T <= bs.FP8_MOE_MAX_TOKENS:
            return bs.fp8_moe_layer(x, w, ids, *self.gate_up, *self.down)
        A, sA = bs.fp8_quantize_tokens(x, rows=token)
        h = torch.empty(T * self.top, self.gate_up[0].shape[1], dtype=torch.bfloat16, device=x.device)
        bs.fp8_gemm_experts(A, sA, *self.gate_up, h, offsets)
        A, sA = bs.fp8_swiglu_quantize_tokens(h)
        y = torch.empty(T * self.top, hidden, dtype=torch.bfloat16, device=x.device)
        bs.fp8_gemm_experts(A, sA, *self.down, y, offsets)
        return (y[places.long()].float() * w[:, :, None]).sum(1).to(torch.bfloat16)

    def reference(self, x):
        """The same layer in fp32 (the same routing and dequantized weights, no FP8 activations)."""
        w, _, offsets, token, places = self.route(x)
        ends = offsets.tolist()
        rows = x.float()[token.long()]
        y = torch.empty(rows.shape, device=x.device)
        up_w, down_w = unpack_weight(*self.gate_up), unpack_weight(*self.down)
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            gate, up = (rows[a:b] @ up_w[e].T).chunk(2, dim=1)
            y[a:b] = (torch.nn.functional.silu(gate) * up) @ down_w[e].T
        return (y[places.long()] * w[:, :, None]).sum(1)


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 512), ("experts", 32), ("top", 4), ("hidden", 2048), ("inner", 1024)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    layer = MoeLayer(a.hidden, a.inner, a.experts, a.top)
    x = torch.randn(a.tokens, a.hidden, generator=torch.Generator(device="cuda").manual_seed(1),
                    device="cuda").to(torch.bfloat16)
    out, ref = layer.forward(x), layer.reference(x)
    err = float((out.float() - ref).norm() / ref.norm())
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        layer.forward(x)
    end.record()
    torch.cuda.synchronize()
    if bs.fp8_status_query() != 0:
        raise RuntimeError("device status set")
    print(f"{a.tokens} tokens, top {a.top} of {a.experts} experts, {a.hidden} -> 2 x {a.inner} -> {a.hidden}: "
          f"relative error {err:.4f} against fp32, {begin.elapsed_time(end) / 20:.3f} ms a layer")


if __name__ == "__main__":
    main()
