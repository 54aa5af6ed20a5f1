"""Attention over the 8-bit paged cache on the GPU against the definition in 64 bits; the tolerances are
derived in cache_q8_ref.attend."""

import math

import pytest
import torch

from cache_q8_ref import Batch, attend, gen

pytestmark = pytest.mark.gpu


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


def queries(batch, Hq, seed, std=1.0):
    return (torch.randn(batch.T, Hq * batch.D, device="cuda", generator=gen(seed)) * std).to(torch.bfloat16)


def check(B, batch, q, cache, scale=None, most=0, table=None, **kw):
    o = torch.full_like(q, 3.5)
    lse = torch.full((batch.T, q.shape[1] // batch.D), 3.5, device="cuda")
    B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, scale=scale, most=most, o=o, lse=lse, **kw)
    want, lwant, bound, lbound = attend(batch, q, cache, batch.D ** -0.5 if scale is None else scale)
    n = sum(batch.new)
    got = o[:n].double().view(n, -1, batch.D)
    off = (got - want[:n]).abs()
    assert (off <= bound[:n]).all(), ((off / bound[:n]).max().item(), int((off > bound[:n]).sum()))
    empty = torch.isinf(lwant[:n])
    assert torch.equal(torch.isinf(lse[:n]) & (lse[:n] < 0), empty)
    loff = (lse[:n].double() - lwant[:n]).abs()
    assert (loff[~empty] <= lbound[:n][~empty]).all(), (loff[~empty] / lbound[:n][~empty]).max().item()
    assert (got[empty] == 0).all()
    assert (o[n:] == 3.5).all() and (lse[n:] == 3.5).all()  # rows behind the last sequence
    clean(B)
    return o


CASES = [  # new, lens, Hq, Hk, D, page
    ([1], [1], 1, 1, 128, 16),
    ([1], [1], 8, 8, 64, 64),
    ([1], [1000], 32, 32, 128, 64),
    ([1, 1, 1, 1], [15, 16, 17, 129], 8, 2, 64, 16),
    ([1] * 40, [1 + 37 * i for i in range(40)], 16, 2, 128, 32),
    ([1], [20001], 8, 1, 128, 64),
    ([1], [7777], 5, 1, 64, 256),
    ([3, 2, 1, 16], [300, 2, 5, 1000], 8, 2, 128, 16),
    ([5] * 9, [100 + 31 * i for i in range(9)], 32, 4, 64, 16),
    ([4, 0, 7, 0], [2, 50, 7, 0], 4, 4, 128, 16),   # padding in front, sequences without rows or tokens
    ([3], [0], 2, 1, 64, 16),                       # rows, but no token at all
    ([17], [17], 4, 2, 128, 16),
    ([33, 1, 64], [40, 500, 640], 12, 4, 128, 64),
    ([127], [127], 1, 1, 128, 128),
    ([128], [256], 8, 8, 64, 64),
    ([129, 300], [129, 433], 8, 2, 128, 16),
    ([257, 1], [2049, 3], 6, 2, 64, 32),
    ([600], [600], 8, 1, 128, 64),
    ([515], [3001], 4, 1, 128, 256),
    ([200, 1, 1, 9], [195, 1000, 70, 9], 16, 4, 128, 64),
    ([90], [333], 7, 1, 64, 16),                    # a group that divides no tile
    ([40], [200], 130, 1, 64, 16),                  # more heads to a key head than a tile has rows
]


@pytest.mark.parametrize("hint", [False, True])
@pytest.mark.parametrize("new,lens,Hq,Hk,D,page", CASES)
def test_attention(B, new, lens, Hq, Hk, D, page, hint):
    batch = Batch(new, lens, Hk, D, page, seed=len(new), extra_rows=2)
    q = queries(batch, Hq, D + len(new), 2.0)
    check(B, batch, q, batch.random_cache(B, seed=3), most=max(new) if hint else 0)


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 40]), ([20, 3], [90, 50]), ([300], [400])])
def test_scores_of_every_size(B, new, lens):
    """One key takes all of the weight, all keys the same weight, and scores that grow along the keys."""
    batch = Batch(new, lens, 2, 128, 16)
    cache = batch.random_cache(B)
    for std, scale in ((40.0, None), (1e-30, None), (0.0, None), (3e37, 1e-37), (1.0, 1e-6), (1.0, 3.0)):
        check(B, batch, queries(batch, 8, 1, std), cache, scale=scale)
    cache[1].copy_(torch.where(cache[1].isnan(), cache[1], torch.linspace(0.001, 0.05, cache[1].numel(), device="cuda")
                               .view_as(cache[1])))
    check(B, batch, queries(batch, 8, 2, 3.0), cache)


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 40]), ([20, 3], [90, 50]), ([300], [400])])
def test_scales_of_every_size(B, new, lens):
    """v's scales over 60 powers of two in one sequence, zeros among them; k's scales zero."""
    batch = Batch(new, lens, 2, 64, 16)
    cache = batch.random_cache(B)
    vs = cache[3]
    power = torch.randint(-40, 21, vs.shape, device="cuda", generator=gen(5)).double()
    vs.copy_(torch.where(power < -35, torch.zeros_like(power), 2.0 ** power).float())
    check(B, batch, queries(batch, 4, 1), cache)
    cache[1].masked_fill_(cache[1] > 0.01, 0.0)
    check(B, batch, queries(batch, 4, 2), cache)
    vs.zero_()
    check(B, batch, queries(batch, 4, 3), cache)


@pytest.mark.parametrize("n", [1, 6, 200])
def test_lost_values_stay_visible(B, n):
    """A NaN or an infinity in a row of q, or a NaN scale, in the rows that see it and in no others."""
    batch = Batch([n, n], [n + 70, n + 90], 2, 128, 16)
    base = batch.random_cache(B)
    q = queries(batch, 8, 1)
    args = (batch.cu, batch.lens, batch.table)
    want = B.coda_attn_q8(q, base, *args)
    for value in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[n, 128 * 3 + 7] = value
        o = B.coda_attn_q8(q2, base, *args).view(2 * n, 8, 128)
        hit = torch.zeros(2 * n, 8, dtype=torch.bool, device="cuda")
        hit[n, 3] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], want.view(2 * n, 8, 128)[~hit])
    for which in (1, 3):
        cache = [t.clone() for t in base]
        pos = batch.total[1] - (n + 1) // 2  # of the second sequence: seen by its last rows
        page, slot = batch.slot(1, pos)
        cache[which][page, 1, slot] = float("nan")
        o = B.coda_attn_q8(q, tuple(cache), *args).view(2 * n, 8, 128)
        hit = torch.zeros(2 * n, 8, dtype=torch.bool, device="cuda")
        hit[2 * n - (n + 1) // 2:, 4:] = True
        assert torch.isnan(o[hit]).all()
        assert not torch.isnan(o[~hit]).any()
        assert (o[~hit].float() - want.view(2 * n, 8, 128)[~hit].float()).abs().max() < 1e-2
    clean(B)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n,group", [(4, 1), (4, 8), (7, 5), (300, 2)])
def test_rows_before_the_first_token_whatever_they_hold(B, n, group, value):
    """Padding in front sees nothing: zeros and -inf, beside rows that see something and in a sequence without a token."""
    batch = Batch([n, 3], [n // 2, 0], 1, 128, 16)
    cache, q = batch.random_cache(B), queries(batch, group, 1)
    bare = n - n // 2
    want, lwant = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, want_lse=True)
    q[:bare, 5::128] = value
    q[n:, 7::128] = value
    o, lse = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, want_lse=True)
    for rows in (slice(0, bare), slice(n, n + 3)):
        assert (o[rows] == 0).all() and (lse[rows] == -float("inf")).all()
    assert torch.equal(o[bare:n], want[bare:n]) and torch.equal(lse[bare:n], lwant[bare:n])
    clean(B)


@pytest.mark.parametrize("n", [1, 6, 200])
def test_bad_pages(B, n):
    batch = Batch([n, n], [n + 70, n + 90], 2, 64, 16)
    cache = batch.random_cache(B)
    q = queries(batch, 4, 1)
    want = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table)
    for value in (-1, batch.pages, 2 ** 31 - 1, -2 ** 31):
        table = batch.table.clone()
        table[1, 2] = value
        o = B.coda_attn_q8(q, cache, batch.cu, batch.lens, table)
        assert B.coda_get_device_status()[1] == 0x240
        assert torch.equal(o[:n], want[:n]) and torch.isnan(o[n:]).all()
    lens = batch.lens.clone()
    lens[1] = batch.table.shape[1] * batch.page + n  # all its rows are beyond the table's end
    o = B.coda_attn_q8(q, cache, batch.cu, lens, batch.table)
    assert B.coda_get_device_status()[1] == 0x240
    assert not torch.isnan(o[:n]).any() and torch.isnan(o[n:]).all()
    lens[1] = 2 ** 31 - 1
    o = B.coda_attn_q8(q, cache, batch.cu, lens, batch.table)
    assert B.coda_get_device_status()[1] == 0x240
    assert torch.isnan(o[n:]).all()
    clean(B)


FEW = [  # new, lens, Hq, Hk, D, page: tiles of 8 rows and of 16, alone and beside sequences of many rows
    ([5, 2, 1], [4000, 129, 77], 16, 4, 128, 64),
    ([2, 1, 1], [6000, 383, 385], 4, 1, 128, 16),
    ([1, 1, 1, 1], [768, 769, 767, 4001], 8, 1, 64, 32),
    ([70, 1, 2, 3], [90, 700, 300, 5000], 16, 1, 128, 32),
    ([70, 1, 2, 3], [90, 700, 300, 5000], 9, 1, 64, 256),
    ([70, 1, 2, 6], [90, 700, 300, 5000], 8, 1, 128, 16),
    ([100, 1, 40, 0, 3], [5000, 1, 2000, 9, 2], 2, 2, 64, 16),
]


@pytest.mark.parametrize("hint", [False, True])
@pytest.mark.parametrize("new,lens,Hq,Hk,D,page", FEW)
def test_attention_of_few_rows(B, new, lens, Hq, Hk, D, page, hint):
    batch = Batch(new, lens, Hk, D, page, seed=len(new), extra_rows=2)
    q = queries(batch, Hq, D + len(new), 2.0)
    check(B, batch, q, batch.random_cache(B, seed=3), most=max(new) if hint else 0)


@pytest.mark.parametrize("new,lens,Hq,Hk,D,page", FEW)
def test_few_rows_same_result_every_time(B, new, lens, Hq, Hk, D, page):
    batch = Batch(new, lens, Hk, D, page)
    cache, q = batch.random_cache(B), queries(batch, Hq, 1, 2.0)
    args = (q, cache, batch.cu, batch.lens, batch.table)
    runs = [B.coda_attn_q8(*args, most=max(new)) for _ in range(60)]
    rows = int(batch.cu[-1])
    assert all(torch.equal(r[:rows], runs[0][:rows]) for r in runs)
    clean(B)


@pytest.mark.parametrize("n", [1, 7, 300])
def test_pages_beyond_2_31_codes(B, n):
    """The same bits as from a small cache with the same two pages."""
    Hk, D, page, g = 8, 128, 256, gen(4)
    pages = (2 ** 31 + 2 ** 28) // (Hk * page * D) + 1
    near = B.coda_cache_q8(2, Hk, page, D)
    for i in (0, 2):
        near[i].copy_(torch.randint(-127, 128, near[i].shape, device="cuda", generator=g))
        near[i + 1].copy_(torch.rand(near[i + 1].shape, device="cuda", generator=g) * 0.02)
    far = B.coda_cache_q8(pages, Hk, page, D)
    for a, b in zip(near, far):
        b[pages - 1] = a[1]
        b[0] = a[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, lens = torch.tensor([0, n], **i32), torch.tensor([300], **i32)
    q = torch.randn(n, 2 * Hk * D, device="cuda", generator=g).to(torch.bfloat16)
    here = B.coda_attn_q8(q, near, cu, lens, torch.tensor([[1, 0]], **i32), want_lse=True)
    there = B.coda_attn_q8(q, far, cu, lens, torch.tensor([[pages - 1, 0]], **i32), want_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(here, there))
    assert torch.isfinite(here[0]).all() and here[0].any()
    clean(B)


SAME = [  # new, lens, Hq, Hk, D, page
    ([1] * 5 + [70], [400, 3000, 17, 900, 5000, 2000], 16, 2, 128, 64),
    ([515], [3001], 4, 1, 128, 256),
    ([515], [3001], 4, 1, 64, 16),
    ([1300], [1300], 8, 8, 128, 64),
]


@pytest.mark.parametrize("new,lens,Hq,Hk,D,page", SAME)
def test_same_result_every_time(B, new, lens, Hq, Hk, D, page):
    """Bit for bit, many times over: a wait that lets something through a moment early shows as a run that differs."""
    batch = Batch(new, lens, Hk, D, page)
    cache, q = batch.random_cache(B), queries(batch, Hq, 1, 2.0)
    args = (q, cache, batch.cu, batch.lens, batch.table)
    runs = [B.coda_attn_q8(*args, most=max(new)) for _ in range(60)]
    assert all(torch.equal(r, runs[0]) for r in runs)
    clean(B)


def test_layer(B):
    """As a model runs it: a chain's y, written to the cache and attended to, chunk by chunk; every chunk's
    result equals the whole prompt's in one call, to the rounding of fp32 sums and of bf16."""
    Hq, Hk, D, page, T = 8, 2, 64, 16, 150
    d = Hq * D
    n1 = (Hq + 2 * Hk) * D
    g = gen(9)
    bf = torch.bfloat16
    x, z = (torch.randn(T, d, device="cuda", generator=g).to(bf) for _ in range(2))
    W0 = (torch.randn(d, d, device="cuda", generator=g) / d ** 0.5).to(bf)
    W1 = (torch.randn(d, n1, device="cuda", generator=g) / d ** 0.5).to(bf)
    gamma = torch.ones(d, device="cuda", dtype=bf)
    _, _, y = B.coda_fwd(x, W0, z, gamma, W1, 1e-5)
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))

    def layer(cuts):
        batch = Batch([T], [T], Hk, D, page)
        cache = B.coda_cache_q8(batch.pages, Hk, page, D)
        out = []
        for a, b in zip(cuts[:-1], cuts[1:]):
            cu, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, b - a], [b]))
            part = y[a:b].contiguous()
            q = B.coda_cache_write_q8(part, cache, cu, lens, batch.table, inv_freq=freq)
            out.append(B.coda_attn_q8(q, cache, cu, lens, batch.table, most=b - a))
        return torch.cat(out), cache

    whole, held = layer([0, T])
    for cuts in ([0, 100, 149, 150], [0, 1, 2, 3, 40, 150], list(range(0, T + 1, 15))):
        parts, cache = layer(cuts)
        k0 = B.coda_cache_read_q8(held, *[torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T], [T])],
                                  Batch([T], [T], Hk, D, page).table, T)
        k1 = B.coda_cache_read_q8(cache, *[torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T], [T])],
                                  Batch([T], [T], Hk, D, page).table, T)
        assert torch.equal(k0[0], k1[0]) and torch.equal(k0[1], k1[1])
        # two results off by 2^-8 of themselves and 2^-10 of the values' size each
        assert ((parts.float() - whole.float()).abs() <= 2 * 2.0 ** -8 * whole.float().abs() + 2 ** -9 * 4).all()
    h, _, y2 = B.coda_fwd(whole, W0, x, gamma, W1, 1e-5)  # the next chain takes it as it is
    assert y2.shape == y.shape and not torch.isnan(y2).any()
    clean(B)
