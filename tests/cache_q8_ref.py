"""The 8-bit paged cache's operators in 64 bits, written out loop by loop, and batches to try them on."""

import math

import torch

U = 2.0 ** -24  # fp32's unit roundoff
UB = 2.0 ** -8  # bf16's
UH = 2.0 ** -11  # fp16's


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Batch:
    """Sequences with `new` rows and `lens` tokens each: cu, lens, a table of shuffled pages (-1 where none
    is needed) of a cache with some spare pages."""

    def __init__(self, new, lens, Hk, D, page, seed=0, spare=3, extra_rows=0):
        g = gen(seed + 1000)
        self.new, self.total, self.Hk, self.D, self.page = list(new), list(lens), Hk, D, page
        need = [-(-max(t, 0) // page) for t in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, device="cuda", generator=g).tolist()
        width = max(max(need, default=0), 1)
        rows, at = [], 0
        for k in need:
            rows.append(order[at:at + k] + [-1] * (width - k))
            at += k
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.tensor(rows, **i32).view(len(rows), width)
        self.cu = torch.tensor([0] + list(torch.tensor(self.new).cumsum(0)), **i32)
        self.lens = torch.tensor(self.total, **i32)
        self.T = sum(self.new) + extra_rows

    def places(self):
        """(row, sequence, token number) of every row of a sequence."""
        row = 0
        for b, (n, t) in enumerate(zip(self.new, self.total)):
            for i in range(n):
                yield row, b, t - n + i
                row += 1

    def slot(self, b, pos):
        return int(self.rows_of_table()[b][pos // self.page]), pos % self.page

    def rows_of_table(self):
        if not hasattr(self, "_rows"):
            self._rows = self.table.tolist()
        return self._rows

    def random_cache(self, B, seed=0, unused=float("nan")):
        """Random codes; scales of slots that hold no token are `unused`."""
        g = gen(seed + 2000)
        cache = B.coda_cache_q8(self.pages, self.Hk, self.page, self.D)
        held = torch.zeros(self.pages, self.page, dtype=torch.bool)
        for b, t in enumerate(self.total):
            for pos in range(max(t, 0)):
                held[self.slot(b, pos)] = True
        for i in (0, 2):
            cache[i].copy_(torch.randint(-128, 128, cache[i].shape, device="cuda", dtype=torch.int8, generator=g))
            cache[i + 1].uniform_(0.002, 0.02, generator=g)
            cache[i + 1].masked_fill_(~held.cuda()[:, None, :], unused)
        return cache

    def tokens(self, codes, scales, b):
        """[tokens, Hk, D] of sequence b in 64 bits."""
        t = max(self.total[b], 0)
        ids = self.table[b, :-(-t // self.page)].long()
        x = codes[ids].double() * scales[ids].double()[..., None]  # [pages, Hk, page, D]
        return x.permute(0, 2, 1, 3).reshape(-1, self.Hk, self.D)[:t]


def attend(batch, q, cache, scale):
    """(o, lse, bound) of q [T, Hq D]: the definition in 64 bits, and how far o may be off.

    A weight's exponent is off by the fp32 sum of D products (one truncation, 2 u, of the running sum
    per 16 of them), five more roundings of numbers up to the largest sum of |q k| of the row, and
    exp2's 2 ulp; its product with v's scale is rounded to fp16 (2^-11, and 2^-25 of the largest
    scale's weight below fp16's range).  Sums of weights times |v| carry these, one truncation of the
    running sum per 16 tokens and the joins of pieces; the result is rounded to bf16."""
    T, n = q.shape
    D, Hk = batch.D, batch.Hk
    Hq = n // D
    o = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    bound, lbound = torch.zeros_like(o), torch.zeros_like(lse)
    at = 0
    for b, (m, t) in enumerate(zip(batch.new, batch.total)):
        if m and t > 0:
            k, v = batch.tokens(*cache[:2], b), batch.tokens(*cache[2:], b)
            k, v = (x.repeat_interleave(Hq // Hk, 1) for x in (k, v))  # a copy of its key head for each query head
            qb = q[at:at + m].double().view(m, Hq, D)
            last = torch.arange(t - m, t, device="cuda")
            unseen = (torch.arange(t, device="cuda") > last[:, None])[:, None, :]
            x = torch.einsum("ihd,jhd->ihj", qb, k) * scale
            size = (torch.einsum("ihd,jhd->ihj", qb.abs(), k.abs()) * scale).masked_fill(unseen, 0.0).amax(2)
            x = x.masked_fill(unseen, -math.inf)
            z = torch.logsumexp(x, 2)
            w = torch.exp(x - torch.where(z > -math.inf, z, torch.zeros_like(z))[:, :, None])
            r = torch.einsum("ihj,jhd->ihd", w, v)
            far = torch.einsum("ihj,jhd->ihd", w, v.abs())
            rel = (2 * (D // 16) + 12) * U * size + 16 * U
            sums = (2 * (t // 16 + 1) + 64) * U
            low = 2.0 ** -25 * t * v.abs().amax((0, 2)) * 2  # [Hq], of weights with maximum one
            top = x.amax(2)
            one = torch.exp(torch.where(z > -math.inf, top - z, torch.zeros_like(z)))  # the largest weight
            o[at:at + m], lse[at:at + m] = r, z
            bound[at:at + m] = UB * r.abs() + (2 * rel + UH + sums)[:, :, None] * 1.05 * far + \
                (low[None] * one)[:, :, None] + 1e-30
            lbound[at:at + m] = rel + sums + 4 * U * z.abs().nan_to_num(0, 0, 0) + 1e-7
        at += m
    return o, lse, bound, lbound


def turn(x, angle, pairs):
    """x [heads, D] (64 bits) with its first 2 len(angle) values turned."""
    out = x.clone()
    half = len(angle)
    for i, a in enumerate(angle):
        j, k = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        out[:, j] = x[:, j] * math.cos(a) - x[:, k] * math.sin(a)
        out[:, k] = x[:, j] * math.sin(a) + x[:, k] * math.cos(a)
    return out
