"""The 8-bit paged cache's calls as programs make them: on other streams, two at once, captured and replayed with
other lengths and pages, with one workspace for two graphs; many sequences; hints that are wrong; and batches that
describe nothing sensible, which may give any rows but touch nothing else and end."""

import pytest
import torch

from cache_q8_ref import Batch, attend, gen
from test_attn_q8_gpu import check, clean, queries

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


def right(batch, q, cache, o):
    want, _, bound, _ = attend(batch, q, cache, batch.D ** -0.5)
    n = sum(batch.new)
    return ((o.double().view(batch.T, -1, batch.D) - want).abs()[:n] <= bound[:n]).all()


def as_int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_another_stream(B):
    batch = Batch([3, 200], [500, 600], 2, 128, 16)
    cache, q = batch.random_cache(B), queries(batch, 8, 1)
    y = torch.randn(batch.T, 12 * 128, device="cuda", generator=gen(2)).to(bf)
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    args = (batch.cu, batch.lens, batch.table)
    want_o = B.coda_attn_q8(q, cache, *args)
    other = [t.clone() for t in cache]
    want_q = B.coda_cache_write_q8(y, other, *args, inv_freq=f)
    want_k, want_v = B.coda_cache_read_q8(other, *args, batch.T)
    mine = [t.clone() for t in cache]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream):
        o = B.coda_attn_q8(q, cache, *args, stream=handle)
        qo = B.coda_cache_write_q8(y, mine, *args, inv_freq=f, stream=handle)
        k, v = B.coda_cache_read_q8(mine, *args, batch.T, stream=handle)
        s.synchronize()
        assert torch.equal(o, want_o) and torch.equal(qo, want_q)
        assert torch.equal(k, want_k) and torch.equal(v, want_v)
    clean(B)


def test_two_streams_at_once(B):
    """Calls of both kernels at the same time, each with its own workspace."""
    jobs = []
    for i, (new, lens, Hq, Hk, D) in enumerate((([1] * 30, [2000 + 50 * j for j in range(30)], 16, 2, 128),
                                                ([700], [900], 8, 2, 64), ([300, 1], [4000, 90], 4, 4, 128))):
        batch = Batch(new, lens, Hk, D, 32, seed=i)
        cache, q = batch.random_cache(B, seed=i), queries(batch, Hq, i)
        want = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table)
        jobs.append((batch, cache, q, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        got = [B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, stream=s) for batch, cache, q, _, s in jobs]
        torch.cuda.synchronize()
        for o, (_, _, _, want, _) in zip(got, jobs):
            assert torch.equal(o, want)
    clean(B)


def test_decoding_from_a_graph(B):
    """One graph of a layer's step, replayed while the sequences grow: lens, the tokens and the pages change under it."""
    Hq, Hk, D, page, n = 8, 2, 64, 16, 3
    lens0 = [5, 31, 200]
    steps = 40
    batch = Batch([1] * n, [t + steps for t in lens0], Hk, D, page)
    cache = Batch([1] * n, lens0, Hk, D, page)  # what is held at first
    held = B.coda_cache_q8(batch.pages, Hk, page, D)
    start = batch.random_cache(B, seed=4, unused=float("nan"))
    for a, b in zip(held, start):
        a.copy_(b)
    y = torch.empty(n, (Hq + 2 * Hk) * D, device="cuda", dtype=bf)
    lens = as_int(lens0)
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    o = torch.empty(n, Hq * D, device="cuda", dtype=bf)
    q = torch.empty_like(o)
    ws = B.workspace(B.coda_attn_q8_workspace_bytes(n, n, Hq, Hk, D), "cuda")

    def step():
        lens.add_(1)
        B.coda_cache_write_q8(y, held, batch.cu, lens, batch.table, inv_freq=freq, q=q)
        B.coda_attn_q8(q, held, batch.cu, lens, batch.table, most=1, o=o, ws=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        lens.copy_(as_int(lens0))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    lens.copy_(as_int(lens0))
    for i in range(steps):
        y.copy_(torch.randn(y.shape, device="cuda", generator=gen(100 + i)))
        g.replay()
        if i % 13 == 0 or i == steps - 1:
            now = Batch([1] * n, [t + i + 1 for t in lens0], Hk, D, page)
            now.table, now._rows = batch.table, batch.table.tolist()
            assert right(now, q, held, o), i
    del cache
    clean(B)


def test_two_graphs_share_a_workspace(B):
    shapes = (([1] * 6, [900 + 77 * i for i in range(6)], 16, 2, 128), ([150, 1], [400, 3000], 16, 2, 128))
    ws = B.workspace(max(B.coda_attn_q8_workspace_bytes(sum(s[0]), len(s[0]), s[2], s[3], s[4]) for s in shapes), "cuda")
    ws.fill_(0xff)
    graphs = []
    for new, lens, Hq, Hk, D in shapes:
        batch = Batch(new, lens, Hk, D, 16)
        cache, q = batch.random_cache(B), queries(batch, Hq, 5)
        want = B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table)
        o = torch.empty_like(want)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            B.coda_attn_q8(q, cache, batch.cu, batch.lens, batch.table, o=o, ws=ws)
        graphs.append((g, o, want, batch, cache, q))
    for _ in range(20):
        for g, o, want, *_ in graphs:
            o.zero_()
            g.replay()
            assert torch.equal(o, want)
    clean(B)


@pytest.mark.parametrize("n", [1000, 8192])
def test_many_sequences(B, n):
    """Short ones; the first and the last have rows for tiles."""
    new, lens = [1] * n, [1 + i % 40 for i in range(n)]
    new[0], lens[0], new[-1], lens[-1], new[7], lens[7] = 70, 90, 60, 64, 0, 5
    batch = Batch(new, lens, 1, 64, 16)
    cache = B.coda_cache_q8(batch.pages, 1, 16, 64)
    g = gen(1)
    for i in (0, 2):
        cache[i].copy_(torch.randint(-128, 128, cache[i].shape, device="cuda", dtype=torch.int8, generator=g))
        cache[i + 1].uniform_(0.002, 0.02, generator=g)
    q = queries(batch, 2, 3)
    check(B, batch, q, cache)
    # the same tokens by one read
    lens_all = as_int([0] + lens).cumsum(0).to(torch.int32)
    k, v = B.coda_cache_read_q8(cache, lens_all, batch.lens, batch.table, sum(lens))
    at = 0
    for b in (0, 1, 7, n // 2, n - 1):
        at = sum(lens[:b])
        assert torch.equal(k[at:at + lens[b]].double(), batch.tokens(*cache[:2], b).to(bf).double()) or \
            (k[at:at + lens[b]].double() - batch.tokens(*cache[:2], b)).abs().max() <= 2.0 ** -7
    clean(B)


@pytest.mark.parametrize("most", [1, 3, 50, 1000])
def test_wrong_hints_change_nothing_but_time(B, most):
    batch = Batch([90, 1, 13], [300, 70, 50], 2, 64, 16)
    check(B, batch, queries(batch, 6, 1), batch.random_cache(B), most=most)


@pytest.mark.parametrize("group,most", [(3, 1), (3, 5), (8, 1), (1, 49)])
def test_wrong_hints_with_items_over_several_blocks(B, group, most):
    # few key heads and many keys: the tiles of the sequence with more rows than the hint says are cut between blocks
    batch = Batch([50, 2], [6001, 900], 1, 64, 16)
    check(B, batch, queries(batch, group, 1), batch.random_cache(B), most=most)


def test_nothing_to_do(B):
    batch = Batch([2], [20], 2, 64, 16)
    cache = batch.random_cache(B)
    empty = torch.empty(0, 4 * 64, device="cuda", dtype=bf)
    cu0, none = as_int([0, 0]), as_int([0])
    assert B.coda_attn_q8(empty, cache, cu0, batch.lens, batch.table).shape == (0, 256)
    assert B.coda_cache_write_q8(torch.empty(0, 8 * 64, device="cuda", dtype=bf), cache, cu0, batch.lens, batch.table).shape == \
        (0, 256)
    assert B.coda_cache_read_q8(cache, cu0, batch.lens, batch.table, 0)[0].shape == (0, 2, 64)
    # rows, but no sequences; sequences, but no rows of theirs
    q = torch.ones(3, 256, device="cuda", dtype=bf)
    o = torch.full_like(q, 3.5)
    B.coda_attn_q8(q, cache, none, as_int([]), torch.empty(0, 1, dtype=torch.int32, device="cuda"), o=o)
    assert (o == 3.5).all()
    B.coda_attn_q8(q, cache, cu0, batch.lens, batch.table, o=o)
    assert (o == 3.5).all()
    clean(B)


NONSENSE = {  # cu, lens of two sequences, 40 rows
    "cu beyond the rows": ([0, 20, 4000], [30, 4010]),
    "cu below zero": ([-5, 20, 40], [30, 30]),
    "cu decreasing": ([0, 30, 10], [40, 40]),
    "cu of the extremes": ([-2 ** 31, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, -2 ** 31]),
    "lens below zero": ([0, 20, 40], [-1, -2 ** 31]),
    "lens beyond the table": ([0, 20, 40], [2 ** 31 - 1, 5000]),
}


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("name", NONSENSE)
def test_nonsense_touches_nothing_else(B, name, group):
    Hk, D, page = 2, 64, 16
    batch = Batch([20, 20], [64, 64], Hk, D, page)
    cu, lens = (as_int(v) for v in NONSENSE[name])
    guard = 64

    def guarded(shape, dtype):  # a tensor inside of a larger one, whose rest must not change
        whole = torch.full((shape[0] + 2 * guard, *shape[1:]), 3, device="cuda", dtype=dtype)
        return whole, whole[guard:-guard]

    q = torch.randn(40, group * Hk * D, device="cuda", generator=gen(1)).to(bf)
    y = torch.randn(40, (group + 2) * Hk * D, device="cuda", generator=gen(2)).to(bf)
    outs = {}
    outs["o"] = guarded(q.shape, bf)
    outs["q"] = guarded(q.shape, bf)
    outs["k"] = guarded((40, Hk, D), bf)
    outs["v"] = guarded((40, Hk, D), bf)
    cache = []
    for i, (shape, dtype) in enumerate((((batch.pages, Hk, page, D), torch.int8), ((batch.pages, Hk, page), torch.float32)) * 2):
        outs[f"cache{i}"] = guarded(shape, dtype)
        cache.append(outs[f"cache{i}"][1])
        cache[-1].fill_(1)
    B.coda_attn_q8(q, cache, cu, lens, batch.table, o=outs["o"][1])
    B.coda_cache_write_q8(y, cache, cu, lens, batch.table, q=outs["q"][1])
    B.coda_cache_read_q8(cache, cu, lens, batch.table, 40, k=outs["k"][1], v=outs["v"][1])
    st, detail = B.coda_get_device_status()
    assert (st, detail) in ((B.CODA_OK, 0), (B.CODA_ERR_DEVICE_BOUNDS, 0x240))
    for n, (whole, _) in outs.items():
        assert (whole[:guard] == 3).all() and (whole[-guard:] == 3).all(), n
    check(B, batch, queries(batch, 4, 1), batch.random_cache(B))  # and the next call is right


@pytest.mark.parametrize("name", ["k_q", "k_s", "v_q", "v_s", "cu", "lens", "table"])
def test_binding_refuses_a_wrong_tensor(B, name):
    batch = Batch([2, 1], [20, 9], 2, 64, 16)
    held = dict(zip(("k_q", "k_s", "v_q", "v_s"), batch.random_cache(B)), cu=batch.cu, lens=batch.lens, table=batch.table)
    right = held[name]
    wide = torch.cat([right, right], -1)
    other = torch.cat([right, right]) if name == "table" else wide  # (a wider table is a right one)
    wrong = [(right.to(torch.int16), TypeError), (right.cpu(), TypeError), (other, ValueError),
             (wide[..., ::2], ValueError)]  # the right shape, every other number
    if name not in ("k_q", "table"):
        wrong.append((right.tolist(), TypeError))
    y, q = torch.zeros(3, 8 * 64, device="cuda", dtype=bf), torch.zeros(3, 4 * 64, device="cuda", dtype=bf)
    for value, error in wrong:
        args = dict(held, **{name: value})
        rest = (tuple(args[n] for n in ("k_q", "k_s", "v_q", "v_s")), args["cu"], args["lens"], args["table"])
        for call in (lambda: B.coda_cache_write_q8(y, *rest), lambda: B.coda_cache_read_q8(*rest, 3),
                     lambda: B.coda_attn_q8(q, *rest)):
            with pytest.raises(error):
                call()
    clean(B)
