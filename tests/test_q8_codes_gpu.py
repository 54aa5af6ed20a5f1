"""Codes and scales of the quantiser against their definition in exact arithmetic.

A bf16 value times 254, and a bf16 amax times an odd number up to 255, are exact in 64 bits, so
  code = rint(127 v / amax), ties to even   <=>   |254 v - 2 code amax| <= amax, the code even where equal
is decided without a rounding.  scale = amax / 127 rounded once to fp32: the quotient in 64 bits is
rounded to 53 bits first, and amax / 127 (period 7 in binary) is never that near to half way
between two fp32 numbers.  No tolerance is left.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 128


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


def check_exact(q, s, x, block):
    M, n = x.shape
    width = block or n
    cut = lambda t: torch.nn.functional.pad(t.double(), (0, -n % width)).view(M, -1, width)  # noqa: E731
    v, code = cut(x), cut(q)
    amax = v.abs().amax(2, keepdim=True)
    off = (254.0 * v - 2.0 * code * amax).abs()
    right = (off < amax) | ((off == amax) & (code % 2 == 0)) | ((amax == 0) & (code == 0))
    assert right.all(), f"{(~right).sum().item()} of {M * n} codes"
    assert torch.equal(s.view(M, -1), (amax.squeeze(2) / 127.0).float())


# a warp's row, a block's row, a row read twice, rows of blocks that walk them
@pytest.mark.parametrize("block", [0, BLOCK])
@pytest.mark.parametrize("M,n", [(300, 128), (257, 264), (64, 1024), (100, 4104), (3, 32776), (650, 16640)])
def test_codes_are_the_definitions(B, M, n, block):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + n)
    x = torch.randn(M, n, device="cuda", generator=g).to(torch.bfloat16)
    check_exact(*B.coda_quant_q8(x, block=block), x, block)


@pytest.mark.parametrize("block", [0, BLOCK])
@pytest.mark.parametrize("exponent", [-125, -108, -20, 0, 93, 120])
def test_every_mantissa_half_way_and_beside(B, exponent, block):
    """Rows whose largest value takes each of the 128 mantissas, with every value of 8 bits, down to
    8 places below the point, beside it: every code half way between two integers that there is,
    and its neighbours.  The exponents reach both ends of bf16's range."""
    top = torch.arange(128, 256, device="cuda", dtype=torch.float64)[:, None]
    step = torch.arange(0, 256, device="cuda", dtype=torch.float64)[None, :]
    v = torch.cat([torch.minimum(step * 2.0 ** -e, top) for e in range(9)], 1)
    v = torch.cat([v, -v], 1)
    v = torch.nn.functional.pad(v, (0, -v.shape[1] % 127)).view(128, -1, 127)
    # the largest value in every block of 128
    x64 = torch.cat([top[:, None].expand(-1, v.shape[1], 1), v], 2).reshape(128, -1) * 2.0 ** exponent
    x = x64.to(torch.bfloat16)
    assert torch.equal(x.double(), x64)
    check_exact(*B.coda_quant_q8(x, block=block), x, block)

