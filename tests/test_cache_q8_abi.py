"""The 8-bit paged cache's checks that need no GPU: refusals that return before anything touches a
device, and the binding's checks."""

import ctypes
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


def _common(p, pages, Hk, page, D, Bn, width, T):
    return (*p[:4], pages, Hk, page, D, *p[4:7], Bn, width, T)


def _write(B, p=(FAKE,) * 9, pages=8, Hk=2, page=16, D=64, Bn=3, width=4, T=5, Hq=4, f=None, axis=None, half=0,
           pos=None, axes=1, pairs=0):
    return B.raw().coda_cache_write_q8(p[7], *_common(p, pages, Hk, page, D, Bn, width, T), Hq, f, axis, half, pos, axes,
                                       pairs, p[8], None)


def _read(B, p=(FAKE,) * 9, pages=8, Hk=2, page=16, D=64, Bn=3, width=4, T=5):
    return B.raw().coda_cache_read_q8(*_common(p, pages, Hk, page, D, Bn, width, T), p[7], p[8], None)


def _attn(B, p=(FAKE,) * 9, pages=8, Hk=2, page=16, D=64, Bn=3, width=4, T=5, Hq=4, scale=0.1, most=0, lse=FAKE, ws=FAKE,
          wsb=BIG):
    return B.raw().coda_attn_q8(p[7], *_common(p, pages, Hk, page, D, Bn, width, T), Hq, scale, most, p[8], lse, ws, wsb,
                                None)


CALLS = {"write": _write, "read": _read, "attn": _attn}


@pytest.mark.parametrize("name", CALLS)
def test_pointers(B, name):
    call = CALLS[name]
    for i in range(9):
        p = [FAKE] * 9
        p[i] = None
        assert call(B, p=p) == B.CODA_ERR_INVALID_ARG, i
        p[i] = FAKE + (2 if 4 <= i < 7 else 8)  # cu, lens and table: 4 bytes
        assert call(B, p=p) == B.CODA_ERR_MISALIGNED, i


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do(B, name):
    assert CALLS[name](B, T=0, p=(None,) * 9) == B.CODA_OK
    assert CALLS[name](B, Bn=0, p=(None,) * 9) == B.CODA_OK


@pytest.mark.parametrize("name", CALLS)
def test_sizes(B, name):
    call = CALLS[name]
    for bad in ({"T": -1}, {"Bn": -1}, {"Hk": 0}, {"D": 0}, {"pages": 0}, {"width": 0}, {"page": 0}, {"page": -16}):
        assert call(B, **bad) == B.CODA_ERR_INVALID_ARG, bad
    for bad in ({"D": 96}, {"D": 256}, {"D": 72}, {"page": 8}, {"page": 48}, {"page": 512}, {"Bn": 8193},
                {"T": 1 << 31}, {"pages": 1 << 31}, {"pages": 1 << 30}, {"width": (1 << 30) // 16 + 1}, {"Hk": 1025}):
        if name != "read" and "Hk" in bad:
            bad["Hq"] = 1025
        assert call(B, **bad) == B.CODA_ERR_UNSUPPORTED_SHAPE, bad
    if name != "read":
        assert call(B, Hq=0) == B.CODA_ERR_INVALID_ARG
        assert call(B, Hq=3) == B.CODA_ERR_UNSUPPORTED_SHAPE  # not a multiple of Hk
        assert call(B, Hq=2048) == B.CODA_ERR_UNSUPPORTED_SHAPE


def test_rotary_arguments(B):
    f = (ctypes.c_double * 32)(*[0.5] * 32)
    a = (ctypes.c_int32 * 32)(*[1] * 32)
    for bad in ({"half": -8, "f": f}, {"half": 8}, {"axes": 0, "pos": FAKE}, {"axes": 5, "pos": FAKE}, {"axes": 2},
                {"half": 8, "f": f, "axis": a}):
        assert _write(B, **bad) == B.CODA_ERR_INVALID_ARG, bad
    for bad in ({"half": 12, "f": f}, {"half": 40, "f": f}):
        assert _write(B, **bad) == B.CODA_ERR_UNSUPPORTED_SHAPE, bad
    assert _write(B, half=8, f=f, pos=FAKE + 2) == B.CODA_ERR_MISALIGNED
    for value in (math.nan, math.inf):
        f[7] = value
        assert _write(B, half=8, f=f, T=0) == B.CODA_ERR_INVALID_ARG
    f[7], a[3] = 0.5, -1
    assert _write(B, half=8, f=f, axis=a, pos=FAKE, axes=2, T=0) == B.CODA_ERR_INVALID_ARG
    a[3] = 1
    assert _write(B, half=8, f=f, axis=a, pos=FAKE, axes=2, T=0) == B.CODA_OK


def test_attention_arguments(B):
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert _attn(B, scale=scale) == B.CODA_ERR_INVALID_ARG
    assert _attn(B, most=-1) == B.CODA_ERR_INVALID_ARG
    need = B.coda_attn_q8_workspace_bytes(5, 3, 4, 2, 64)
    assert need > 0
    assert _attn(B, wsb=need - 1) == B.CODA_ERR_WORKSPACE_TOO_SMALL
    assert _attn(B, ws=None) == B.CODA_ERR_WORKSPACE_TOO_SMALL
    assert _attn(B, ws=FAKE + 8) == B.CODA_ERR_MISALIGNED
    assert _attn(B, lse=FAKE + 4) == B.CODA_ERR_MISALIGNED
    for bad in ((0, 3, 4, 2, 64), (5, 0, 4, 2, 64), (5, 3, 4, 3, 64), (5, 3, 4, 2, 80), (-1, 3, 4, 2, 64)):
        assert B.coda_attn_q8_workspace_bytes(*bad) == 0


def test_binding_refuses_before_any_launch(B):
    cache = tuple(torch.zeros(s, dtype=t) for s, t in (((4, 2, 16, 64), torch.int8), ((4, 2, 16), torch.float32)) * 2)
    cu, lens, table = torch.tensor([0, 1], dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    bf = torch.bfloat16
    with pytest.raises(ValueError):  # heads of 64 values
        B.coda_cache_write_q8(torch.zeros(1, 100, dtype=bf), cache, cu, lens, table)
    with pytest.raises(ValueError):  # no query head
        B.coda_cache_write_q8(torch.zeros(1, 256, dtype=bf), cache, cu, lens, table)
    with pytest.raises(ValueError):
        B.coda_attn_q8(torch.zeros(1, 100, dtype=bf), cache, cu, lens, table)
    for call in (lambda: B.coda_cache_write_q8(torch.zeros(1, 512, dtype=bf), cache, cu, lens, table),
                 lambda: B.coda_cache_read_q8(cache, cu, lens, table, 1),
                 lambda: B.coda_attn_q8(torch.zeros(1, 256, dtype=bf), cache, cu, lens, table)):
        with pytest.raises(TypeError):  # not CUDA tensors
            call()
    with pytest.raises(TypeError):
        B._host(torch.zeros(4), torch.float64, 4, "inv_freq")
    with pytest.raises(ValueError):
        B._host(torch.zeros(4, dtype=torch.int32), torch.int32, 8, "axis")
