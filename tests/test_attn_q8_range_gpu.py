"""Attention over the 8-bit paged cache at the ends of its numeric range, on the GPU against the definition in 64 bits.

The tolerances are cache_q8_ref.attend's unless a test says otherwise."""

import math

import pytest
import torch

from cache_q8_ref import U, UB, UH, Batch, attend, gen
from test_attn_q8_gpu import check, clean, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


SHAPES = [  # new, lens, Hq, Hk, D: tiles of 8 rows, of 16, and of 256
    ([1, 1], [1000, 37], 4, 2, 128),
    ([5, 1], [1003, 60], 8, 2, 64),
    ([200, 3], [900, 300], 4, 1, 128),
]


# ------------------------------------------------------------------ large value scales
@pytest.mark.parametrize("power", [60, 100, 115, 121, 126])
@pytest.mark.parametrize("new,lens,Hq,Hk,D", SHAPES)
def test_large_value_scales(B, new, lens, Hq, Hk, D, power):
    """Whatever v's scales, a row's weights and their sum are the scores': o is the definition's and lse does not
    change.  (The codes keep o within fp32.)"""
    batch = Batch(new, lens, Hk, D, 16)
    cache = batch.random_cache(B)
    q = queries(batch, Hq, power, 2.0)
    _, lse = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, want_lse=True)
    most = 2 if power > 121 else 63
    cache[2].clamp_(-most, most)
    cache[3].mul_(50.0).mul_(2.0 ** power)  # 2^power times 0.1 to 1
    check(B, batch, q, cache)
    _, lse2 = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, want_lse=True)
    # two lse of the same scores, whose sums may be taken in other units: each off by its sum's rounding
    t = max(lens)
    assert ((lse - lse2).abs() <= 2 * (2 * (t // 16 + 1) + 64) * U + 8 * U * lse.abs()).all()


def test_the_largest_values_that_a_write_keeps(B):
    """Values near bf16's end through the cache: what is read back, attended to, is its mean."""
    T, Hk, D = 300, 1, 64
    batch = Batch([T], [T], Hk, D, 16)
    y = torch.randn(T, 3, D, device="cuda", generator=gen(1))
    y[:, 2] = (torch.rand(T, D, device="cuda", generator=gen(2)) * 2 - 1) * 3e38
    y = y.to(torch.bfloat16).view(T, -1)
    cache = B.coda_cache_q8(batch.pages, Hk, 16, D)
    q = B.coda_cache_write_q8(y, cache, batch.cu, batch.lens, batch.table)
    assert cache[3][batch.table[0, 0].long()].amax() > 2.0 ** 119
    check(B, batch, q, cache)


# ------------------------------------------------------------------ tokens that a row does not see
@pytest.mark.parametrize("value", [2.0 ** 12, 2.0 ** 20, 2.0 ** 100, 2.0 ** 121, float("inf"), float("nan")])
@pytest.mark.parametrize("new,lens,Hq,Hk,D", [([5, 1], [1003, 60], 8, 2, 64), ([6, 1], [30, 9], 8, 8, 128),
                                              ([200, 1], [900, 30], 4, 1, 128), ([330, 70], [330, 2000], 2, 2, 64)])
def test_scales_of_unseen_tokens(B, new, lens, Hq, Hk, D, value):
    """Rows before a token give the same bits whatever that token's v scale is."""
    batch = Batch(new, lens, Hk, D, 16)
    cache, q = batch.random_cache(B), queries(batch, Hq, 3, 2.0)
    args = (q, cache, batch.cu, batch.lens, batch.table)
    o, lse = B.coda_attn_q8(*args, want_lse=True)
    for back in (1, 2, new[0] // 2):  # the last token, the last but one, one in the middle
        page, slot = batch.slot(0, lens[0] - back)
        was = cache[3][page, :, slot].clone()
        cache[3][page, :, slot] = value
        o2, lse2 = B.coda_attn_q8(*args, want_lse=True)
        cache[3][page, :, slot] = was
        before, behind = slice(0, new[0] - back), slice(new[0], None)
        for rows in (before, behind):
            assert torch.equal(o2[rows], o[rows]) and torch.equal(lse2[rows], lse[rows])
        assert torch.equal(lse2, lse)  # which knows no v
        seen = o2[new[0] - back:new[0]]
        assert not torch.equal(seen, o[new[0] - back:new[0]])
    clean(B)


# ------------------------------------------------------------------ many small weights
@pytest.mark.parametrize("n,group,seqs", [(1, 1, 1), (2, 8, 1), (60, 1, 160)])
@pytest.mark.parametrize("bits,steps", [(17.0, 106.5), (17.5, 75.5), (18.0, 53.5), (18.5, 40.5)])
def test_many_small_weights_beside_a_large_one(B, n, group, seqs, bits, steps):
    """A first token of weight one and 131072 others of weight 2^-bits each, alike, with values of the other sign: what
    their weights lose together is within fp16's 2^-11 of each.  (`steps`: their weight times scale in steps of 2^-24 if
    the first one's is near one: midway between two.)  160 sequences of the same pages, so that whole rows of keys are one
    block's.

    The bound, relative to the sum of |weights times values|, which is v: as attend's for scores of size bits log 2,
    without a term for what lies below fp16's range; and o's rounding."""
    t, D = 131072 + n, 64
    pages = -(-t // 256)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(pages, device="cuda", generator=gen(1)).to(torch.int32)
    k_q, k_s, v_q, v_s = cache = B.coda_cache_q8(pages, 1, 256, D)
    k_q.zero_()
    k_s.fill_(1.0 / 64)
    v_q.fill_(100)
    v_s.fill_(steps * 2.0 ** (bits - 24) * 2.0 ** -6)
    first = int(table[0])
    k_q[first, 0, 0] = 64
    v_q[first, 0, 0] = -100
    q = torch.zeros(seqs * n, group, D, device="cuda", dtype=torch.bfloat16)
    q[:, :, 5] = 16.0
    size = bits * math.log(2)
    o = B.coda_attn_q8(q.view(seqs * n, -1), cache, torch.arange(seqs + 1, device="cuda", dtype=torch.int32) * n,
                       torch.full((seqs,), t, **i32), table.repeat(seqs, 1), scale=size / 16, most=n)
    others = torch.arange(t - n, t, device="cuda").double().repeat(seqs)  # that each row sees
    small = math.exp(-16 * torch.tensor(size / 16, dtype=torch.float32).item())
    v = 100 * v_s[0, 0, 0].item()
    want = (v * (others * small - 1) / (1 + others * small))[:, None]
    rel = (2 * (D // 16) + 12) * U * size + 16 * U
    sums = (2 * (t // 16 + 1) + 64) * U
    off = (o.double() - want).abs()
    bound = UB * want.abs() + (2 * rel + UH + sums) * 1.05 * v
    assert (off <= bound).all(), (off / bound).max().item()
    clean(B)


# ------------------------------------------------------------------ one sequence in many batches
def exact_scores(B, n, t, Hq, Hk, D, seed):
    """A sequence whose scores are multiples of 1/4 in base 2 and whose weighted sums of codes are exact in fp32, so that
    nothing but the weights' rounding to fp16, relative to a power of two, and a last rounding of a quotient is left.
    (q, codes, scales, scale) and the definition with its weights rounded so."""
    g = gen(seed)
    q = torch.zeros(n, Hq, D, device="cuda")
    q[:, :, :2] = torch.tensor([1.0, 0.25], device="cuda")
    q[:, :, 2] = torch.randint(0, 2, (n, Hq), device="cuda", generator=g).float()
    k = torch.zeros(t, Hk, D, dtype=torch.int8, device="cuda")
    k[:, :, 0] = torch.randint(-1, 2, (t, Hk), device="cuda", generator=g).to(torch.int8)
    k[:, :, 1] = torch.randint(-2, 3, (t, Hk), device="cuda", generator=g).to(torch.int8)
    k[:, :, 2] = torch.randint(0, 2, (t, Hk), device="cuda", generator=g).to(torch.int8)
    # values that go by the fraction of a score (k's second column), so that its weights' roundings do not average out
    sign = torch.randint(-1, 2, (5, D), device="cuda", generator=g).to(torch.int8)
    v = sign[k[:, :, 1].long() + 2]
    # a scale whose product with log2 e is one in fp32
    e = torch.tensor(1.44269504088896, dtype=torch.float32)
    near = [torch.tensor(math.log(2), dtype=torch.float32) + i * 2.0 ** -24 for i in range(-4, 5)]
    scale = next(float(s) for s in near if s * e == 1.0)
    group = Hq // Hk
    x = torch.einsum("ihd,jhd->ihj", q.double(), k.double().repeat_interleave(group, 1))
    unseen = (torch.arange(t, device="cuda") > torch.arange(t - n, t, device="cuda")[:, None])[:, None]
    w = torch.exp2(x).masked_fill(unseen, 0.0)
    # fp16 has 11 bits: its rounding of a number between two powers of two
    unit = torch.exp2(torch.floor(x) - 10)
    frac = w / unit
    assert ((frac - frac.floor() - 0.5).abs() > 2.0 ** -8)[~unseen.expand_as(frac)].all()  # none near a tie
    w16 = torch.round(frac) * unit
    vv = v.double().repeat_interleave(group, 1)
    o = torch.einsum("ihj,jhd->ihd", w16.masked_fill(unseen, 0.0), vv) / w.sum(2)[..., None]
    return q.to(torch.bfloat16).view(n, -1), k, v, scale, o


@pytest.mark.parametrize("most", [0, 1, 1000])
@pytest.mark.parametrize("others", [[], [(1, 5000)] * 3, [(1, 700)] * 40, [(300, 900)], [(77, 300), (1, 9), (2, 4000), (500, 500)]])
@pytest.mark.parametrize("n,t,Hq,Hk,D", [(1, 300, 4, 2, 128), (3, 257, 8, 2, 64), (90, 300, 2, 2, 128), (70, 200, 4, 1, 64)])
def test_one_sequence_in_many_batches(B, n, t, Hq, Hk, D, others, most):
    """Other sequences and the hint decide where a sequence's keys are cut and which kernel takes it; its weights round the
    same way all the same.  Off by fp32 rounding alone: the sum of weights and the quotient (t + 64 roundings of the
    result), the parts and their joins (24 and 160 of numbers up to 0.25); then bf16's, which keeps order: what lies
    between two numbers before it lies between their roundings behind it."""
    q1, k, v, scale, want = exact_scores(B, n, t, Hq, Hk, D, 7)
    new, lens = [m for m, _ in others], [m for _, m in others]
    at = len(others) // 2
    new.insert(at, n)
    lens.insert(at, t)
    batch = Batch(new, lens, Hk, D, 16)
    cache, q = batch.random_cache(B), queries(batch, Hq, 5)
    row = sum(new[:at])
    q[row:row + n] = q1
    ids, slot = batch.table[at, torch.arange(t, device="cuda") // 16].long(), torch.arange(t, device="cuda") % 16
    cache[0][ids, :, slot], cache[1][ids, :, slot] = k, 1.0
    cache[2][ids, :, slot], cache[3][ids, :, slot] = v, 0.25
    o = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, scale=scale, most=most)
    got, want = o[row:row + n].view(n, Hq, D), want * 0.25
    slack = ((t + 64) * want.abs() + (24 + 160) * 0.25) * U
    low, high = (want - slack).float().to(torch.bfloat16), (want + slack).float().to(torch.bfloat16)
    assert ((got >= low) & (got <= high)).all(), int(((got < low) | (got > high)).sum())
    clean(B)


# ------------------------------------------------------------------ large scores
@pytest.mark.parametrize("scale", [3e5, 1e7, 1e8, 7e8, 1e10, 3e15])
@pytest.mark.parametrize("new,lens,Hq,Hk,D", SHAPES)
def test_large_scores(B, new, lens, Hq, Hk, D, scale):
    """Scores that fp32 holds to whole numbers or worse: whichever keys win, the outputs are means of their values.  All
    values of a head are the same, so o is: off by the weights' rounding, which its sum does not have (2^-11), the sums'
    (t / 16 truncations, joins) and bf16's.  lse is the largest score, to the rounding of a score (rel of attend)."""
    batch = Batch(new, lens, Hk, D, 16)
    cache = batch.random_cache(B)
    cache[2].copy_(torch.arange(D, device="cuda") % 101 - 50)
    cache[3].fill_(0.25)
    cache[0][:, :, 8:].copy_(cache[0][:, :, :8].clone())  # pairs of keys with one score
    cache[1][:, :, 8:].copy_(cache[1][:, :, :8].clone())
    q = queries(batch, Hq, 3, 2.0)
    o, lse = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, scale=scale, want_lse=True)
    want = ((torch.arange(D, device="cuda") % 101 - 50) * 0.25).double()
    t = max(lens)
    slack = (UH + (2 * (t // 16 + 1) + 64) * U) * 1.05 + UB
    assert ((o.double().view(batch.T, Hq, D) - want).abs() <= slack * want.abs()).all()
    _, lwant, _, lbound = attend(batch, q, cache, scale)
    assert ((lse.double() - lwant).abs() <= lbound).all()
    clean(B)
