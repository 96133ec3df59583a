"""Chains of the 128-granular calls, each reading what the one before it wrote, with every
buffer rewritten in place: enqueued back to back (the kernels overlap by programmatic
dependent launch) they give the bits of the same chain with a synchronisation after each call."""
import pytest
import torch

from tests._block128 import blocks

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bs():
    import block_scaled_fp8_sm_gb300 as mod
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    mod.library()
    return mod


def _weights(E, N, K, g):
    q = torch.randn(E, N, K, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.exp2(torch.randint(-1, 1, (E, blocks(N), blocks(K)), generator=g, device=DEV).float()
                   - torch.log2(torch.tensor(float(K))).item() // 2)
    return q, s


class Chain:
    """`steps` layers x -> experts -> gate -> experts -> x over preallocated buffers."""

    def __init__(self, bs, T, hidden, inner, E, mode=None, dense=False):
        g = torch.Generator(device=DEV).manual_seed(T + hidden)
        self.bs, self.mode, self.dense = bs, mode, dense
        self.x0 = torch.randn(T, hidden, generator=g, device=DEV).to(torch.bfloat16)
        self.up, self.down = _weights(E, 2 * inner, hidden, g), _weights(E, hidden, inner, g)
        cuts = torch.sort(torch.randint(0, T + 1, (E - 1,), generator=g, device=DEV)).values
        self.off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
        self.rows = torch.randperm(T, generator=g, device=DEV).to(torch.int32)
        u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
        make = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device=DEV)   # noqa: E731
        self.x = make(T, hidden, dtype=bf)
        self.A, self.sA = make(T, hidden, dtype=u8), make(T, blocks(hidden), dtype=f32)
        self.h = make(T, 2 * inner, dtype=bf)
        self.G, self.sG = make(T, inner, dtype=u8), make(T, blocks(inner), dtype=f32)

    def product(self, A, sA, W, C):
        if self.dense:
            return self.bs.fp8_gemm_block128(A, sA, W[0][0], W[1][0], C, mode=self.mode)
        return self.bs.fp8_gemm_experts(A, sA, *W, C, self.off, mode=self.mode)

    def run(self, steps, lead=None, wait=False):
        self.x.copy_(self.x0)
        if lead is not None:
            lead()
        pow2 = self.mode == self.bs.FP8_PATH_NATIVE
        calls = (lambda: self.bs.fp8_quantize_tokens(self.x, self.A, self.sA, rows=self.rows, pow2=pow2),
                 lambda: self.product(self.A, self.sA, self.up, self.h),
                 lambda: self.bs.fp8_swiglu_quantize_tokens(self.h, self.G, self.sG, pow2=pow2),
                 lambda: self.product(self.G, self.sG, self.down, self.x))
        for _ in range(steps):
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [t.clone() for t in (self.x, self.A, self.sA, self.h, self.G, self.sG)]


# rows form; split tiles; tiles; the block-scaled MMA; one dense product after another
CASES = [(1, 512, 256, 4, None, False), (24, 512, 384, 16, None, False), (60, 2064, 1040, 3, None, False),
         (700, 528, 400, 8, None, False), (5000, 1040, 528, 2, 1, False), (5, 1040, 528, 1, None, True),
         (40, 2064, 528, 1, None, True), (3000, 1296, 784, 1, 1, True), (300, 528, 272, 1, 2, True)]


@pytest.mark.parametrize("lead", ["sleep", "product"])
@pytest.mark.parametrize("T,hidden,inner,E,mode,dense", CASES)
def test_back_to_back_equals_synchronised(bs, T, hidden, inner, E, mode, dense, lead):
    chain = Chain(bs, T, hidden, inner, E, mode, dense)
    want = chain.run(6, wait=True)
    assert bool(torch.isfinite(want[0].float()).all()) and bool((want[0] != 0).any())
    if lead == "sleep":   # the whole chain is enqueued before its first kernel starts
        first = lambda: torch.cuda._sleep(4_000_000)   # noqa: E731
    else:                 # a long product on some of the SMs: the chain's first kernels wait beside it
        K = 65536
        q = torch.zeros(5120, K, dtype=torch.uint8, device=DEV)
        s, w = torch.ones(5120, K // 128, device=DEV), torch.zeros(64, K, dtype=torch.uint8, device=DEV)
        out = torch.empty(5120, 64, dtype=torch.bfloat16, device=DEV)
        first = lambda: bs.fp8_gemm_block128(q, s, w, s[:1], out, mode=bs.FP8_PATH_PROMOTE)   # noqa: E731
    for _ in range(4):
        got = chain.run(6, first)
        for name, a, b in zip(("x", "A", "sA", "h", "G", "sG"), got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    assert bs.fp8_status_query() == 0
