"""The 8-bit paged cache on the GPU: writing with rotary positions and reading back, against the
definition in 64 bits.

Tolerances (u = 2^-24 fp32's, 2^-8 bf16's unit roundoff):
  turned values  cos and sin within 2 ulp and the angle's rounding to fp32 (pi u): 6 u each; two
                 products and a sum more: |a| + |b| times 8 u.
  codes          the quotient by amax of a turned value: |a| + |b| is at most twice the head's amax
                 (a pair keeps its length), so the code is off by 127 * (2 * 2 * 8 + 4) u < 3e-4 before it is
                 rounded.  A value that is not turned is a bf16 number, whose code is the definition's.
  scales         amax / 127: 4 u of it, and a turned amax's 16 u.
  values read    bf16(code * scale): the same two roundings as in torch: equal.
"""

import math

import pytest
import torch

from cache_q8_ref import U, UB, Batch, gen, turn

pytestmark = pytest.mark.gpu
CODES = 3e-4


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


def clean(B):
    st, detail = B.coda_get_device_status()
    assert st == B.CODA_OK, (B.status_string(st), hex(detail))


def blank(B, batch):
    """A cache in which every slot can be told to be untouched."""
    cache = B.coda_cache_q8(batch.pages, batch.Hk, batch.page, batch.D)
    for i in (0, 2):
        cache[i].fill_(77)
        cache[i + 1].fill_(-5.0)
    return cache


def rows(batch, Hq, seed):
    y = torch.randn(batch.T, Hq + 2 * batch.Hk, batch.D, device="cuda", generator=gen(seed)) * 2
    y[:, :, 3] *= 9
    return y.view(batch.T, -1).to(torch.bfloat16)


def freqs(half, theta=10000.0):
    return theta ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))


def check_written(B, batch, cache, y, q, angles, half, pairs):
    """Everything that a write may and may not have done.  angles[row]: the row's angles."""
    Hk, D = batch.Hk, batch.D
    Hq = y.shape[1] // D - 2 * Hk
    y64 = y.double().cpu().view(batch.T, -1, D)
    host = [c.cpu() for c in cache]
    qh = q.double().cpu().view(batch.T, Hq, D)
    left = torch.ones(batch.pages, batch.page, dtype=torch.bool)
    for row, b, pos in batch.places():
        x = y64[row].clone()
        x[:Hq + Hk] = turn(x[:Hq + Hk], angles[row], pairs)
        both = torch.zeros_like(x)  # |a| + |b| of the pair
        if half:
            size = y64[row].abs()
            if pairs:
                two = size[:, 0:2 * half:2] + size[:, 1:2 * half:2]
                both[:, :2 * half] = two.repeat_interleave(2, 1)
            else:
                two = size[:, :half] + size[:, half:2 * half]
                both[:, :2 * half] = torch.cat((two, two), 1)
        assert ((qh[row] - x[:Hq]).abs() <= UB * x[:Hq].abs() + 8 * U * both[:Hq] * (1 + UB)).all(), row
        if pos < 0:
            continue
        page, slot = batch.slot(b, pos)
        left[page, slot] = False
        for i, part in ((0, x[Hq:Hq + Hk]), (2, x[Hq + Hk:])):
            amax = part.abs().amax(1)
            exact = part * torch.where(amax > 0, 127 / amax, torch.zeros_like(amax))[:, None]
            turned = i == 0 and half > 0
            codes = host[i][page, :, slot].double()
            assert ((codes - exact).abs() <= 0.5 + (CODES if turned else 1e-9)).all(), (row, i)
            got, want = host[i + 1][page, :, slot].double(), amax / 127
            assert ((got - want).abs() <= (20 if turned else 4) * U * want).all(), (row, i)
    for i in (0, 2):  # nothing else was touched
        assert (host[i].permute(0, 2, 1, 3)[left] == 77).all()
        assert (host[i + 1].permute(0, 2, 1)[left] == -5.0).all()


SHAPES = [  # new, lens, Hq, Hk, D, page
    ([1], [1], 1, 1, 128, 16),
    ([1], [1001], 32, 32, 128, 64),
    ([1, 1, 1], [5, 16, 17], 8, 2, 64, 16),
    ([7, 0, 1, 33], [7, 3, 90, 40], 6, 2, 128, 32),
    ([5, 20], [3, 300], 5, 5, 64, 256),       # two rows of the first stand before its first token
    ([0, 130, 0], [0, 131, 9], 28, 4, 64, 16),
    ([1] * 70, list(range(1, 71)), 2, 1, 128, 16),  # more sequences than a warp has lanes
    ([1300], [1311], 3, 1, 64, 128),          # four tokens to a block, the last block ragged
]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("part", [0, 0.5, 0.75, 1])
@pytest.mark.parametrize("new,lens,Hq,Hk,D,page", SHAPES)
def test_write(B, new, lens, Hq, Hk, D, page, part, pairs):
    batch = Batch(new, lens, Hk, D, page, extra_rows=2)
    half = int(D * part) // 2
    y = rows(batch, Hq, len(new) + D)
    cache, q = blank(B, batch), torch.full((batch.T, Hq * D), 3.5, device="cuda", dtype=torch.bfloat16)
    f = freqs(half)
    B.coda_cache_write_q8(y, cache, batch.cu, batch.lens, batch.table, inv_freq=f if half else None, pairs=pairs,
                          q=q)
    angles = {row: [pos * w for w in f.tolist()] for row, _, pos in batch.places()}
    check_written(B, batch, cache, y, q, angles, half, pairs)
    assert (q[sum(new):] == 3.5).all()  # rows behind the last sequence
    k, v = (torch.full((batch.T, Hk, D), 3.5, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    B.coda_cache_read_q8(cache, batch.cu, batch.lens, batch.table, batch.T, k=k, v=v)
    check_read(batch, cache, k, v)
    clean(B)


def check_read(batch, cache, k, v):
    for row, b, pos in batch.places():
        for out, i in ((k, 0), (v, 2)):
            if pos < 0:
                assert (out[row] == 0).all()
                continue
            page, slot = batch.slot(b, pos)
            want = (cache[i][page, :, slot].float() * cache[i + 1][page, :, slot, None]).to(torch.bfloat16)
            assert torch.equal(out[row], want), (row, i)
    n = sum(batch.new)
    assert (k[n:] == 3.5).all() and (v[n:] == 3.5).all()


@pytest.mark.parametrize("axes", [2, 3, 4])
def test_positions_on_several_axes(B, axes):
    batch = Batch([40, 1], [60, 9], 2, 64, 16)
    half, Hq = 24, 4
    y = rows(batch, Hq, axes)
    axis = (torch.arange(half) * axes // half).to(torch.int32)
    axis[5] = axes - 1  # in any order
    pos = torch.randint(-50, 5000, (axes, batch.T), device="cuda", dtype=torch.int32, generator=gen(axes))
    f = freqs(half, 500.0)
    cache = blank(B, batch)
    q = B.coda_cache_write_q8(y, cache, batch.cu, batch.lens, batch.table, inv_freq=f, axis=axis, pos=pos)
    at = pos.tolist()
    angles = {row: [at[a][row] * w for a, w in zip(axis.tolist(), f.tolist())] for row, _, _ in batch.places()}
    check_written(B, batch, cache, y, q, angles, half, False)
    clean(B)


def test_far_positions(B):
    """Positions up to 2^31 - 1 and below zero; frequencies of every size and sign."""
    batch = Batch([9], [9], 1, 64, 16)
    f = freqs(32)
    f[3], f[4], f[5], f[6] = 7.25, -0.125, 0.0, 100.0
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 12345678, -7, 0, 1, 99999999, 2 ** 24 + 1]],
                       device="cuda", dtype=torch.int32)
    y = rows(batch, 2, 5)
    cache = blank(B, batch)
    q = B.coda_cache_write_q8(y, cache, batch.cu, batch.lens, batch.table, inv_freq=f, pos=pos)
    # (a 64-bit product of a far position keeps 22 bits below one: the remainder by 2 pi is exact there)
    angles = {}
    for row in range(9):
        p = int(pos[0, row])
        angles[row] = [math.remainder(p * w, 2 * math.pi) for w in f.tolist()]
    check_far(batch, y, q, angles)
    clean(B)


def check_far(batch, y, q, angles):
    y64, qh = y.double().cpu().view(batch.T, -1, 64), q.double().cpu().view(batch.T, 2, 64)
    for row in range(batch.T):
        want = turn(y64[row][:2], angles[row], False)
        size = y64[row][:2].abs()
        both = torch.cat((size[:, :32] + size[:, 32:],) * 2, 1)
        # the reference's own product and its remainder: 2^31 * 100 * 2^-53 and the 2 pi of 2^-52 relative
        slack = 1e-4
        assert ((qh[row] - want).abs() <= UB * want.abs() + (8 * U + slack) * both).all(), row


def test_extreme_values(B):
    batch = Batch([6], [6], 1, 64, 16)
    y = torch.zeros(6, 3, 64, device="cuda")
    y[0] = 2.0 ** -133
    y[1] = 3.0e38
    y[2, :, 5] = float("inf")
    y[3, :, 7] = float("nan")
    y[4, :, 0] = -1.0
    y = y.to(torch.bfloat16).view(6, -1)
    cache = blank(B, batch)
    q = B.coda_cache_write_q8(y, cache, batch.cu, batch.lens, batch.table)
    assert torch.equal(q.nan_to_num(7), y.view(6, 3, 64)[:, 0].nan_to_num(7))
    k, v = B.coda_cache_read_q8(cache, batch.cu, batch.lens, batch.table, 6)
    for out in (k, v):
        x = y.view(6, 3, 64)[:, 0].double()
        got = out[:, 0].double()
        assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
        for r in (0, 1, 4, 5):
            step = x[r].abs().max() / 127
            assert ((got[r] - x[r]).abs() <= 0.5 * step + UB * x[r].abs() + 2.0 ** -134).all(), r
    clean(B)


def bad_tables(batch):
    """(table, the sequence and the tokens that it loses)"""
    for value in (-1, batch.pages, 2 ** 31 - 1, -2 ** 31):
        t = batch.table.clone()
        t[1, 1] = value
        yield t, 1, range(batch.page, min(2 * batch.page, batch.total[1]))


def test_bad_pages_are_not_touched(B):
    batch = Batch([20, 40], [20, 60], 2, 64, 16)
    y = rows(batch, 2, 1)
    for table, seq, lost in bad_tables(batch):
        good, cache = blank(B, batch), blank(B, batch)
        B.coda_cache_write_q8(y, good, batch.cu, batch.lens, batch.table)
        clean(B)
        B.coda_cache_write_q8(y, cache, batch.cu, batch.lens, table)
        st, detail = B.coda_get_device_status()
        assert (st, detail) == (B.CODA_ERR_DEVICE_BOUNDS, 0x240)
        page = int(batch.table[seq, 1])
        for a, b in zip(good, cache):
            want = a.clone()
            want[page] = 77 if a.dtype == torch.int8 else -5.0
            assert torch.equal(b, want)
        k, v = B.coda_cache_read_q8(good, batch.cu, batch.lens, table, batch.T)
        assert B.coda_get_device_status()[1] == 0x240
        for row, b, pos in batch.places():
            assert torch.isnan(k[row]).all().item() == (b == seq and pos in lost)
            assert torch.isnan(v[row]).all().item() == (b == seq and pos in lost)
    # a sequence longer than its row of the table
    lens = batch.lens.clone()
    lens[1] = batch.table.shape[1] * batch.page + 5
    k, _ = B.coda_cache_read_q8(good, batch.cu, lens, batch.table, batch.T)
    assert B.coda_get_device_status()[1] == 0x240
    assert torch.isnan(k[-5:]).all() and not torch.isnan(k[-6]).any()
    clean(B)


def test_more_than_2_31_codes(B):
    """Pages whose codes lie beyond 2^31 bytes."""
    Hk, D, page = 8, 128, 256
    pages = (2 ** 31 + 2 ** 28) // (Hk * page * D) + 1
    cache = B.coda_cache_q8(pages, Hk, page, D)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 0]], **i32)
    cu, lens = torch.tensor([0, 300], **i32), torch.tensor([300], **i32)
    y = (torch.randn(300, 3 * Hk * D, device="cuda", generator=gen(3))).to(torch.bfloat16)
    B.coda_cache_write_q8(y, cache, cu, lens, table)
    k, v = B.coda_cache_read_q8(cache, cu, lens, table, 300)
    x = y.view(300, 3, Hk, D).float()
    for out, i in ((k, 1), (v, 2)):
        step = x[:, i].abs().amax(2, keepdim=True) / 127
        assert ((out.float() - x[:, i]).abs() <= 0.501 * step + UB * x[:, i].abs()).all()
    clean(B)
