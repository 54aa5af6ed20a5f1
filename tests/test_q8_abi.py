"""The 8-bit operators' checks that need no GPU: refusals that return before anything touches
a device, workspace sizes, and the binding's checks of blocks."""

import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

FAKE = 0x10000  # a 16-byte-aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    return binding


def _quant(B, M=4, n=64, block=0, p=(FAKE,) * 3):
    return B.raw().coda_quant_q8(p[0], M, n, block, p[1], p[2], None)


def _dequant(B, M=4, n=64, block=0, p=(FAKE,) * 3):
    return B.raw().coda_dequant_q8(p[0], p[1], M, n, block, p[2], None)


def _norm(B, M=4, d=64, eps=1e-5, p=(FAKE,) * 6):
    return B.raw().coda_add_rmsnorm_q8(p[0], p[1], p[2], eps, M, d, p[3], p[4], p[5], None)


def _product(B, M=4, K=64, N=64, p=(FAKE,) * 6, ws=FAKE, wsb=BIG):
    return B.raw().coda_matmul_q8(p[0], p[1], p[2], p[3], p[4], M, K, N, p[5], ws, wsb, None)


def _bwd(B, M=4, d=64, N1=64, Dout=64, p=(FAKE,) * 12, ws=FAKE, wsb=BIG):
    return B.raw().coda_bwd_swiglu_dgrad_q8(*p[:8], M, d, N1, Dout, *p[8:], ws, wsb, None)


CALLS = {"quant": (_quant, 3, ()), "dequant": (_dequant, 3, ()), "norm": (_norm, 6, (1, 3)),
         "product": (_product, 6, (4,)), "bwd": (_bwd, 12, (11,))}


@pytest.mark.parametrize("name", CALLS)
def test_pointers_are_checked(B, name):
    call, count, optional = CALLS[name]
    for i in range(count):
        if i not in optional:
            p = [FAKE] * count
            p[i] = None
            assert call(B, p=p) == B.CODA_ERR_INVALID_ARG, i
        p = [FAKE] * count
        p[i] = FAKE + 8
        assert call(B, p=p) == B.CODA_ERR_MISALIGNED, i


@pytest.mark.parametrize("name", CALLS)
def test_rows(B, name):
    call, count, _ = CALLS[name]
    assert call(B, M=-1) == B.CODA_ERR_INVALID_ARG
    assert call(B, M=1 << 31) == B.CODA_ERR_UNSUPPORTED_SHAPE
    assert call(B, M=0, p=[None] * count) == B.CODA_OK  # empty batch: no-op


def test_sizes_that_overflow_are_refused(B):
    """Within the limit of each size, but with more values than any device holds."""
    lim = (1 << 31) - 256
    assert _quant(B, M=lim, n=lim // 8 * 8) == B.CODA_ERR_UNSUPPORTED_SHAPE
    assert _dequant(B, M=lim, n=lim // 8 * 8, block=128) == B.CODA_ERR_UNSUPPORTED_SHAPE
    assert _norm(B, M=lim, d=lim // 8 * 8) == B.CODA_ERR_UNSUPPORTED_SHAPE
    top = lim // 16 * 16
    for M, K, N in ((1, top, top), (lim, top, 16), (lim, 16, top)):
        assert _product(B, M=M, K=K, N=N) == B.CODA_ERR_UNSUPPORTED_SHAPE
        assert B.coda_matmul_q8_workspace_bytes(M, K, N) == 0


@pytest.mark.parametrize("call", [_quant, _dequant], ids=["quant", "dequant"])
def test_quantiser_shapes(B, call):
    assert call(B, n=0) == B.CODA_ERR_INVALID_ARG
    assert call(B, n=12) == B.CODA_ERR_UNSUPPORTED_SHAPE
    assert call(B, n=1 << 31) == B.CODA_ERR_UNSUPPORTED_SHAPE
    for block in (-1, 1, 64, 256):
        assert call(B, block=block) == B.CODA_ERR_INVALID_ARG


def test_norm_shapes_and_eps(B):
    assert _norm(B, d=-8) == B.CODA_ERR_INVALID_ARG
    assert _norm(B, d=20) == B.CODA_ERR_UNSUPPORTED_SHAPE
    for eps in (-1.0, math.nan, math.inf):
        assert _norm(B, eps=eps) == B.CODA_ERR_INVALID_ARG


def test_product_shapes_and_workspace(B):
    assert _product(B, K=0) == B.CODA_ERR_INVALID_ARG
    assert _product(B, N=-16) == B.CODA_ERR_INVALID_ARG
    for bad in ({"K": 24}, {"N": 40}, {"K": 1 << 31}, {"N": 1 << 31}):
        assert _product(B, **bad) == B.CODA_ERR_UNSUPPORTED_SHAPE
    for M, K, N in ((1, 16, 16), (32, 8192, 8192), (1024, 4096, 4096)):  # up to 1024 tokens: none
        assert B.coda_matmul_q8_workspace_bytes(M, K, N) == 0
        assert _product(B, M, K, N, ws=FAKE + 4) == B.CODA_ERR_MISALIGNED
    for M, K, N in ((1025, 16, 16), (2048, 1040, 784), (8192, 4096, 28672)):
        need = B.coda_matmul_q8_workspace_bytes(M, K, N)
        assert need > 0
        assert _product(B, M, K, N, wsb=need - 1) == B.CODA_ERR_WORKSPACE_TOO_SMALL
        assert _product(B, M, K, N, ws=None) == B.CODA_ERR_WORKSPACE_TOO_SMALL
        assert _product(B, M, K, N, ws=FAKE + 4) == B.CODA_ERR_MISALIGNED
    assert B.coda_matmul_q8_workspace_bytes(0, 64, 64) == 0
    assert B.coda_matmul_q8_workspace_bytes(4, 24, 64) == 0


def test_backward_shapes_and_workspace(B):
    for bad in ({"N1": 0}, {"d": 0}, {"Dout": 0}):
        assert _bwd(B, **bad) == B.CODA_ERR_INVALID_ARG
    # rows of N1 / 2 codes start on 16-byte boundaries
    for bad in ({"N1": 48}, {"d": 12}, {"Dout": 20}):
        assert _bwd(B, **bad) == B.CODA_ERR_UNSUPPORTED_SHAPE
    need = B.coda_bwd_swiglu_dgrad_workspace_bytes(4, 64, 64, 64)
    assert _bwd(B, wsb=need - 1) == B.CODA_ERR_WORKSPACE_TOO_SMALL
    assert _bwd(B, ws=FAKE + 8) == B.CODA_ERR_MISALIGNED


def test_binding_refuses_before_any_launch(B):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        B.coda_quant_q8(x, block=64)
    with pytest.raises(ValueError):
        B.coda_dequant_q8(q, torch.zeros(4), block=32)
    with pytest.raises(ValueError):
        B.coda_add_rmsnorm_q8(x, x[0], 1e-5, h=x)
    with pytest.raises(TypeError):
        B.coda_quant_q8(x)  # not a CUDA tensor
