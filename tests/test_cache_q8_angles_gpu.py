"""The angles of the 8-bit cache's rotary positions, near and far, against exact ones.

Values are made to cancel: of bf16's numbers a = m 2^-7, b = n 2^-7 (m, n of 8 bits) those two whose ratio is nearest to
the angle's tangent, so that a cos t - b sin t is some 2^-15 of them and the rounding of the result to bf16 hides nothing.

Tolerance: cos and sin within 2 ulp each, two products and a sum, (|a| + |b|) 8 u as in test_cache_q8_gpu; and beside that
the angle's own rounding to 2^-26 of a turn and what is cut off its 32 bits and its products, 2^-31 of a turn."""

import math
from fractions import Fraction

import pytest
import torch

from cache_q8_ref import U, UB, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


def two_pi(bits=256):
    """2 pi in steps of 2^-bits: 8 (4 arctan(1/5) - arctan(1/239)) ... of Machin."""
    one = 1 << (bits + 32)

    def arctan_inverse(x):
        total, power, k = 0, one // x, 1
        while power:
            total += power // k if k % 4 == 1 else -(power // k)
            power //= x * x
            k += 2
        return total

    return 8 * (4 * arctan_inverse(5) - arctan_inverse(239)) >> 32


def exact_angle(pos, freq, bits=256):
    """pos * freq less whole turns, between -pi and pi, to a double's rounding."""
    turn = two_pi(bits)
    at = Fraction(freq) * pos * (1 << bits)
    rest = (at.numerator // at.denominator) % turn
    if rest > turn // 2:
        rest -= turn
    return rest / (1 << bits)


def cancelling(angle):
    """(a, b) of eight bits each with the smallest a cos - b sin."""
    c, s = math.cos(angle), math.sin(angle)
    best = min(((abs(m * abs(c) - n * abs(s)), m, n) for m in range(64, 256)
                for n in ([round(m * abs(c / s))] if s and 64 <= m * abs(c / s) <= 255 else [])), default=None)
    if best is None:  # near an axis: no such ratio
        return (1.0, 1.0)
    _, m, n = best
    return m / 128, math.copysign(n / 128, c * s)


POSITIONS = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 12345678, -7, 0, 1, 99999999, 2 ** 24 + 1, 131071, -2 ** 28 - 3]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("freqs", [
    [1.0, 0.5, 0.1, 1 / 3, 7.25, -0.125, 100.0, 0.01],
    [1000.0, -12345.678, 1e6, 2.0 ** 32 / 3, 1e-3, 1e-6, -1.0, 3.0],
    [10000.0 ** (-i / 8) for i in range(8)],
])
def test_angles_at_any_position(B, freqs, pairs):
    half, D = 8, 64
    n = len(POSITIONS)
    batch = Batch([n], [n], 1, D, 16)
    pos = torch.tensor([POSITIONS], device="cuda", dtype=torch.int32)
    angles = [[exact_angle(p, f) for f in freqs] for p in POSITIONS]
    y = torch.zeros(n, 3, D, dtype=torch.float64)
    first = [2 * i for i in range(half)] if pairs else list(range(half))
    second = [i + 1 if pairs else i + half for i in first]
    for r in range(n):
        for i in range(half):
            y[r, :2, first[i]], y[r, :2, second[i]] = cancelling(angles[r][i])
    yb = y.to(torch.bfloat16)
    assert torch.equal(yb.double(), y)
    cache = B.coda_cache_q8(batch.pages, 1, 16, D)
    q = B.coda_cache_write_q8(yb.view(n, -1).cuda(), cache, batch.cu, batch.lens, batch.table,
                              inv_freq=torch.tensor(freqs, dtype=torch.float64), pos=pos, pairs=pairs)
    got = q.double().cpu().view(n, D)
    worst = 0.0
    for r in range(n):
        for i in range(half):
            a, b = y[r, 0, first[i]].item(), y[r, 0, second[i]].item()
            c, s = math.cos(angles[r][i]), math.sin(angles[r][i])
            want = a * c - b * s, a * s + b * c
            for w, at in zip(want, (first[i], second[i])):
                slack = UB * abs(w) + (8 * U + 2 * math.pi * (2.0 ** -26 + 2.0 ** -31)) * (abs(a) + abs(b))
                worst = max(worst, abs(got[r, at].item() - w) / slack)
    assert worst <= 1.0, worst
    st, detail = B.coda_get_device_status()
    assert st == B.CODA_OK, (B.status_string(st), hex(detail))
