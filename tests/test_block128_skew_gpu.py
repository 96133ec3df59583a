"""Few rows over many experts, unevenly: the rows form, with up to 500 rows for one expert."""
import itertools

import pytest
import torch

from tests._accept import bf16_to_f64, check
from tests._block128 import Product, product

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bs():
    import block_scaled_fp8_sm_gb300 as mod
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    mod.library()
    return mod


def _counts(E, **rows):
    c = [0] * E
    for e, n in rows.items():
        c[int(e[1:])] = n
    return c


@pytest.mark.parametrize("counts", [
    _counts(64, e5=256), _counts(64, e0=33, e1=32, e31=31, e32=65, e63=64), _counts(40, e0=1, e7=97, e39=2),
    _counts(8, e7=32), _counts(9, e0=33), _counts(300, e3=500, e127=1, e128=129, e129=33, e299=400),
    [1] * 31 + [70] + [1] * 32,
])
def test_an_expert_has_most_of_the_rows(bs, counts):
    E, N, K = len(counts), 40, 272
    T = sum(counts)
    assert T <= 4 * E   # the rows form
    p = Product(T, N, K, seed=E, E=E)
    off = [0] + list(itertools.accumulate(counts))
    C = torch.full((T + 1, N), -7.0, dtype=torch.bfloat16, device=DEV)
    bs.fp8_gemm_experts(*p.on(DEV), C[:T], torch.tensor(off, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert bs.fp8_status_query() == 0 and bool((C[T] == -7.0).all())
    got = bf16_to_f64(C)
    for e, c in enumerate(counts):
        if c:
            r = slice(off[e], off[e + 1])
            Cr, Tm = product(p.A[r], p.sA[r], p.B[e], p.sB[e])
            check(got[r], Cr, Tm, f"skewed experts {E} e{e}")
