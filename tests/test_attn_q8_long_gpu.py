"""Attention over the 8-bit paged cache where it is long: items cut over many blocks, pages looked up over many units, sums
over many moves of what is taken out of the exponents.  Tolerances as in cache_q8_ref.attend, whose terms for sums grow with
the number of keys; against the definition in 64 bits."""

import pytest
import torch

from cache_q8_ref import Batch
from test_attn_q8_gpu import check, clean, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


LONG = [  # new, lens, Hq, Hk, D, page
    ([8192], [8192], 4, 4, 128, 64),            # a whole prompt
    ([5003, 3151], [5003, 3151], 4, 2, 64, 16),  # two packed
    ([700, 1], [30000, 9000], 4, 1, 128, 256),  # a chunk far into a context, beside a token
    ([4097], [12289], 2, 2, 64, 32),            # a tile's last row by itself, a unit's first key by itself
    ([1, 2], [131072, 40001], 8, 1, 64, 128),   # few rows, cut over all blocks
]


@pytest.mark.parametrize("new,lens,Hq,Hk,D,page", LONG)
def test_long(B, new, lens, Hq, Hk, D, page):
    batch = Batch(new, lens, Hk, D, page, seed=len(new), extra_rows=3)
    check(B, batch, queries(batch, Hq, D, 2.0), batch.random_cache(B, seed=3), most=max(new))


@pytest.mark.parametrize("n,t", [(3000, 6000), (6, 20000)])
def test_scores_that_grow_along_the_keys(B, n, t):
    """Each key's score above the last one's: what is taken out of the exponents moves all the way."""
    batch = Batch([n], [t], 1, 128, 16)
    cache = batch.random_cache(B)
    where = torch.arange(t, device="cuda")
    page, slot = batch.table[0, where // 16].long(), where % 16
    cache[0][page, 0, slot] = 0
    cache[0][page, 0, slot, 7] = 127
    cache[1][page, 0, slot] = torch.linspace(0.0, 0.1, t, device="cuda")
    cache[3][page, 0, slot] = torch.logspace(-4, -1, t, device="cuda")  # v's scales too
    q = torch.zeros(n, 2, 128, device="cuda")
    q[:, :, 7] = torch.tensor([100.0, 400.0], device="cuda")  # 112 and 449 in all, 0.02 to 0.07 a key
    check(B, batch, q.to(torch.bfloat16).view(n, -1), cache)
    clean(B)
