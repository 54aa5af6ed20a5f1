"""What the 8-bit paged cache's binding refuses before any launch; needs no GPU."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    return binding


def test_a_cache_of_heads_without_values(B):
    """D = 0 is refused as other values that heads cannot have, not by a division."""
    cache = B.coda_cache_q8(4, 2, 16, 0, device="cpu")
    cu, lens, table = (torch.zeros(s, dtype=torch.int32) for s in ((2,), (1,), (1, 1)))
    for call in (B.coda_cache_write_q8, B.coda_attn_q8):
        with pytest.raises(ValueError, match="heads of 0 values"):
            call(torch.zeros(1, 64, dtype=torch.bfloat16), cache, cu, lens, table)
