"""The 8-bit paged cache's operators as their users call them: cases, plain forms and 64-bit values.

  write  coda_cache_write_q8: a projection's rows [q | k | v] are split, q and k turned by their
         rotary positions (one axis, or several for images and video), k and v written to the pages
         as INT8 codes with one scale per token and head; then coda_cache_read_q8 of the same tokens
  read   coda_cache_read_q8: whole sequences out of their pages, in bf16
  attn   coda_attn_q8: attention of each sequence's new tokens over its part of the cache, causal,
         with shared key and value heads; one token, a few, a chunk or a whole prompt

`run` calls the framework's entry points where `own` is set, and computes the plain form in
elementary torch operations in 32 bits otherwise; `exact` computes the definition in 64 bits.
"""

import math

import torch

own = False


def listed():
    return [
        # one token of a 7B-class model (32 heads, none shared) while decoding
        {"name": "write_token", "op": "write", "seqs": 1, "new": 1, "held": 1000, "ones": 0, "Hq": 32, "Hk": 32,
         "D": 128, "page": 64, "axes": 1, "rot": 128, "pairs": False, "empty": 0},
        # a prompt with an image: three axes, a part of the head turned, an odd number of tokens
        {"name": "write_image", "op": "write", "seqs": 3, "new": 1531, "held": 70, "ones": 1, "Hq": 28, "Hk": 4,
         "D": 64, "page": 16, "axes": 3, "rot": 48, "pairs": True, "empty": 2},
        # a prompt of 8192 tokens at 70B-class head counts, far into a long context
        {"name": "write_prompt", "op": "write", "seqs": 1, "new": 8192, "held": 100000, "ones": 0, "Hq": 64, "Hk": 8,
         "D": 128, "page": 64, "axes": 1, "rot": 128, "pairs": False, "empty": 0},
        # a batch of ragged sequences of small heads handed over to another worker
        {"name": "read_ragged", "op": "read", "seqs": 9, "new": 1, "held": 700, "Hq": 8, "Hk": 4, "D": 64, "page": 16,
         "empty": 0},
        # a long context read back whole
        {"name": "read_long", "op": "read", "seqs": 2, "new": 1, "held": 40000, "Hq": 32, "Hk": 8, "D": 128, "page": 128,
         "empty": 0},
        # one token of a 7B-class model over a short context: latency
        {"name": "attn_token", "op": "attn", "seqs": 1, "new": 1, "held": 999, "ones": 0, "Hq": 32, "Hk": 32, "D": 128,
         "page": 64, "lse": False, "empty": 0},
        # a decoding batch at 70B-class head counts, every sequence at its own length
        {"name": "attn_decode", "op": "attn", "seqs": 64, "new": 1, "held": 8191, "ones": 0, "Hq": 64, "Hk": 8, "D": 128,
         "page": 64, "lse": False, "empty": 0},
        # one token at the end of a long document
        {"name": "attn_long", "op": "attn", "seqs": 1, "new": 1, "held": 131071, "ones": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "lse": True, "empty": 0},
        # drafted tokens of a speculating batch checked together, small heads
        {"name": "attn_drafts", "op": "attn", "seqs": 16, "new": 5, "held": 3000, "ones": 0, "Hq": 32, "Hk": 4, "D": 64,
         "page": 16, "lse": False, "empty": 0},
        # two chunks of prompts beside four decoding sequences, one of the chunks padded in front
        {"name": "attn_chunk", "op": "attn", "seqs": 6, "new": 509, "held": 8192, "ones": 4, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "lse": True, "empty": 3},
        # two whole prompts packed one after the other
        {"name": "attn_prompts", "op": "attn", "seqs": 2, "new": 5003, "held": 0, "ones": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "lse": False, "empty": 0},
        # a whole prompt of 8192 tokens
        {"name": "attn_prompt", "op": "attn", "seqs": 1, "new": 8192, "held": 0, "ones": 0, "Hq": 32, "Hk": 32, "D": 128,
         "page": 64, "lse": False, "empty": 0},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "read", "attn", "attn", "attn"))
    D = rng.choice((64, 128, 128))
    Hk = rng.choice((1, 2, 4, 8, 8, 32))
    Hq = Hk * rng.choice((1, 2, 4, 5, 8) if Hk <= 8 else (1,))
    c = {"op": op, "Hq": Hq, "Hk": Hk, "D": D, "page": rng.choice((16, 32, 64, 128, 256)), "empty": 0}
    if op == "write":
        seqs = _spread(rng, 1, 64)
        c.update(seqs=seqs, new=_spread(rng, 1, 8192 // seqs), held=_spread(rng, 1, 100000), axes=rng.choice((1, 1, 2, 3)),
                 rot=rng.choice((D, D, D // 2, 3 * D // 4)), pairs=rng.random() < 0.4)
        c["ones"] = rng.randint(0, seqs - 1) if rng.random() < 0.3 else 0
        while seqs * c["held"] > 400000:
            c["held"] //= 2
    elif op == "read":
        seqs = _spread(rng, 1, 32)
        c.update(seqs=seqs, new=1, held=_spread(rng, 15, 60000 // seqs))
    else:
        kind = rng.choice(("token", "few", "chunk", "prompt"))
        if kind == "token":
            seqs, new, held = _spread(rng, 1, 128), 1, _spread(rng, 1, 100000)
        elif kind == "few":
            seqs, new, held = _spread(rng, 1, 32), rng.randint(2, 16), _spread(rng, 1, 32768)
        elif kind == "chunk":
            seqs, new, held = _spread(rng, 1, 8), _spread(rng, 17, 1024), _spread(rng, 64, 16384)
        else:
            seqs, new, held = rng.randint(1, 4), _spread(rng, 17, 6000), 0
        while seqs * held > 200000 or seqs * Hq * new * (new + held) > 32 * 8192 * 6000:
            held, new = held // 2, max(1, new * 3 // 4)
        c.update(seqs=seqs, new=new, held=held, lse=rng.random() < 0.4)
        c["ones"] = rng.randint(0, seqs - 1) if rng.random() < 0.3 else 0
    if op != "read" and c["new"] > 8 and rng.random() < 0.3:
        c["empty"] = rng.randint(1, 5)
    return c


def lengths(case):
    """The new tokens of each sequence and its tokens in all: every sequence its own, the first the
    longest, the last `ones` of them with a single new token.  The first `empty` new tokens of the
    first sequence are padding: they stand before its first position."""
    new, total = [], []
    for b in range(case["seqs"]):
        one = b >= case["seqs"] - case.get("ones", 0)
        n = 1 if one else max(1, round(case["new"] * (1 - 0.6 * (b * 0.618034 % 1))))
        held = round(case["held"] * (1 - 0.8 * (b * 0.754878 % 1)))
        if b == 0 and case["empty"]:
            held = -min(case["empty"], n)
        new.append(n)
        total.append(n + held)
    if case["op"] == "read":
        new = total
    return new, total


# --------------------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)


def _codes(gen, shape):
    """Codes of a quantised bell-shaped tensor: most small, the largest at the range's end."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in out.view(-1).split(1 << 26):
        part.copy_(_normal(gen, part.shape, 32.0).round_().clamp_(-127, 127))
    return out


def _cache(gen, case, total):
    """Pages in a shuffled order, a table of them (-1 where a sequence has none), and the cache; the
    slots that hold no token have a scale of NaN, as memory that nothing has written may."""
    Hk, D, page = case["Hk"], case["D"], case["page"]
    used = [-(-max(n, 0) // page) for n in total]
    pages = sum(used) + 3
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    at = torch.arange(max(max(used), 1), device="cuda")[None, :]
    count = torch.tensor(used, device="cuda")[:, None]
    first = torch.cumsum(count, 0) - count
    table = torch.where(at < count, order[(first + at).clamp_max(pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    cache = []
    for _ in range(2):
        scales = torch.rand((pages, Hk, page), device="cuda", generator=gen) * 0.02 + 0.02
        cache += [_codes(gen, (pages, Hk, page, D)), scales]
    place = torch.arange(at.numel() * page, device="cuda")[None, :]
    seq, pos = (place < torch.tensor(total, device="cuda")[:, None]).nonzero(as_tuple=True)
    held = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
    held[table[seq, pos // page].long(), pos % page] = True
    for scales in cache[1::2]:
        scales.masked_fill_(~held[:, None, :], float("nan"))
    return table.contiguous(), cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    s = dict(case)
    new, total = lengths(case)
    T = sum(new)
    s["rows"], s["most"] = T, max(new)
    s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    s["lens"] = torch.tensor(total, device="cuda", dtype=torch.int32)
    s["table"], s["cache"] = _cache(gen, case, total)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "write":
        y = _normal(gen, (T, Hq + 2 * Hk, D))
        y[:, :, torch.randint(0, D, (2,), device="cuda", generator=gen)] *= 8.0  # loud channels
        s["y"] = y.view(T, -1).to(torch.bfloat16)
        half = case["rot"] // 2
        s["inv_freq"] = 500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        s["pos"], s["axis"] = None, None
        if case["axes"] > 1:  # time, height and width of patches: one position on each axis
            s["axis"] = (torch.arange(half) * case["axes"] // half).to(torch.int32)
            s["pos"] = torch.randint(0, 4000, (case["axes"], T), device="cuda", generator=gen, dtype=torch.int32)
    elif case["op"] == "attn":
        s["q"] = _normal(gen, (T, Hq * D), 2.0).to(torch.bfloat16)
    return s


# --------------------------------------------------------------------------- one pass
def _places(s):
    """Of each row: its sequence, its position there, its page and its slot in the page."""
    row = torch.arange(s["rows"], device="cuda")
    cu, lens = s["cu"].long(), s["lens"].long()
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = lens[seq] - (cu[seq + 1] - row)
    at = pos.clamp_min(0)
    return pos, s["table"][seq, at // s["page"]].long(), at % s["page"]


def _plain_read(s, places):
    pos, page, slot = places
    gone = (pos < 0)[:, None, None]
    k_q, k_s, v_q, v_s = s["cache"]
    k = k_q[page, :, slot].float() * k_s[page, :, slot][:, :, None]
    v = v_q[page, :, slot].float() * v_s[page, :, slot][:, :, None]
    zero = torch.zeros((), device="cuda")
    return {"k": torch.where(gone, zero, k).to(torch.bfloat16), "v": torch.where(gone, zero, v).to(torch.bfloat16)}


def _plain_turn(x, cos, sin, pairs):
    """x [T, heads, D]: the first 2 * cos.shape[1] values of a head as pairs (i, i + half), or
    (2 i, 2 i + 1) with `pairs`, each turned by its angle."""
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    head, rest = x[:, :, :2 * half], x[:, :, 2 * half:]
    if pairs:
        a, b = head[:, :, 0::2], head[:, :, 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), 3).flatten(2)
    else:
        a, b = head[:, :, :half], head[:, :, half:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), 2)
    return torch.cat((turned, rest), 2)


def _plain_codes(u):
    amax = u.abs().amax(2, keepdim=True)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(u * inv).to(torch.int8), (amax / 127.0).squeeze(2)


def _plain_write(s):
    Hq, Hk, D = s["Hq"], s["Hk"], s["D"]
    pos, page, slot = places = _places(s)
    at = pos[None, :] if s["pos"] is None else s["pos"].long()
    axis = torch.zeros(s["rot"] // 2, dtype=torch.long) if s["axis"] is None else s["axis"].long()
    angle = at[axis.cuda()].t().double() * s["inv_freq"].cuda()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    y = s["y"].float().view(-1, Hq + 2 * Hk, D)
    q, k = _plain_turn(y[:, :Hq], cos, sin, s["pairs"]), _plain_turn(y[:, Hq:Hq + Hk], cos, sin, s["pairs"])
    real = pos >= 0
    (kq, ks), (vq, vs) = _plain_codes(k[real]), _plain_codes(y[:, Hq + Hk:][real])
    page, slot = page[real], slot[real]
    s["cache"][0][page, :, slot], s["cache"][1][page, :, slot] = kq, ks
    s["cache"][2][page, :, slot], s["cache"][3][page, :, slot] = vq, vs
    return dict(_plain_read(s, places), q=q.flatten(1).to(torch.bfloat16))


def _plain_attn(s):
    Hq, Hk, D, page = s["Hq"], s["Hk"], s["D"], s["page"]
    group, B = Hq // Hk, s["seqs"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"]
    n, width = cu[1:] - cu[:-1], table.shape[1] * page
    key = torch.arange(width, device="cuda")
    held = (key < lens[:, None])[:, None, :, None]  # [B, 1, width, 1]
    pages = table.clamp_min(0).long()
    zero = torch.zeros((), device="cuda")

    def gather(codes, scales):
        wide = codes[pages].transpose(1, 2).reshape(B, Hk, width, D).float()
        return torch.where(held, wide * scales[pages].transpose(1, 2).reshape(B, Hk, width, 1), zero)

    k, v = gather(*s["cache"][:2]), gather(*s["cache"][2:])
    i = torch.arange(s["most"], device="cuda")
    real = i < n[:, None]
    row = (cu[:-1, None] + i).clamp_max(s["rows"] - 1)
    q = s["q"].float()[row].view(B, -1, Hk, group, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    score = (q @ k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hk, group, -1, width)
    last = (lens - n)[:, None] + i  # the last key that a new token sees
    seen = (key <= last[:, :, None])[:, None, None]
    score = score.masked_fill_(~seen, float("-inf"))
    top = score.amax(4, keepdim=True)
    top = torch.where(top == float("-inf"), zero, top)
    p = score.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    o = (p.view(B, Hk, -1, width) @ v).view(B, Hk, group, -1, D) / torch.where(total > 0, total, torch.ones_like(total))
    out = {"o": o.permute(0, 3, 1, 2, 4).reshape(B, -1, Hq * D)[real].to(torch.bfloat16)}
    if s["lse"]:
        out["lse"] = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, -1, Hq)[real]
    return out


def run(s):
    if not own:
        return _plain_write(s) if s["op"] == "write" else _plain_read(s, _places(s)) if s["op"] == "read" else _plain_attn(s)
    from gemm_epilogue_fusion_gemm0_gb300 import binding as B

    batch = (s["cache"], s["cu"], s["lens"], s["table"])
    if s["op"] == "read":
        k, v = B.coda_cache_read_q8(*batch, s["rows"])
        return {"k": k, "v": v}
    if s["op"] == "write":
        q = B.coda_cache_write_q8(s["y"], *batch, inv_freq=s["inv_freq"], axis=s["axis"], pos=s["pos"], pairs=s["pairs"])
        k, v = B.coda_cache_read_q8(*batch, s["rows"])
        return {"q": q, "k": k, "v": v}
    if s["lse"]:
        o, lse = B.coda_attn_q8(s["q"], *batch, most=s["most"], want_lse=True)
        return {"o": o, "lse": lse}
    return {"o": B.coda_attn_q8(s["q"], *batch, most=s["most"])}


# --------------------------------------------------------------------------- work
def work(case):
    new, total = lengths(case)
    Hq, Hk, D, T = case["Hq"], case["Hk"], case["D"], sum(new)
    entry = 2 * Hk * (D + 4)  # a token of the cache: codes and scales of k and v
    small = 4 * (3 * case["seqs"] + sum(-(-max(n, 0) // case["page"]) for n in total))
    if case["op"] == "read":
        return {"bytes": T * (entry + 4 * Hk * D) + small, "flops": 2 * T * Hk * D}
    if case["op"] == "write":  # rows in; q, the cache's entries, and the values read back out
        pos = 4 * T * case["axes"] if case["axes"] > 1 else 0
        return {"bytes": T * (2 * (Hq + 2 * Hk) * D + 2 * Hq * D + entry + 4 * Hk * D) + pos + small,
                "flops": T * (3 * (Hq + Hk) * case["rot"] + 8 * Hk * D)}
    pairs = 0
    for n, t in zip(new, total):  # keys seen by the new tokens: t - n + 1 .. t, none of them below 0
        m = min(n, max(t, 0))
        pairs += m * t - m * (m - 1) // 2
    return {"bytes": sum(max(t, 0) for t in total) * entry + 4 * T * Hq * D + (4 * T * Hq if case["lse"] else 0) + small,
            "flops": 4 * pairs * Hq * D}


# --------------------------------------------------------------------------- 64 bits
def _sequence(s, b, total):
    """k and v of a sequence, [Hk, tokens, D]: its pages one after the other."""
    count = -(-total // s["page"])
    ids = s["table"][b, :count].long()

    def values(codes, scales):
        x = codes[ids].double() * scales[ids].double().unsqueeze(3)
        return torch.cat(list(x), 1)[:, :total]

    return values(*s["cache"][:2]), values(*s["cache"][2:])


def _exact_turn(head, angle, pairs):
    half = angle.shape[1]
    first = torch.arange(half, device="cuda") * 2 if pairs else torch.arange(half, device="cuda")
    second = first + (1 if pairs else half)
    z = torch.complex(head[:, first], head[:, second]) * torch.polar(torch.ones_like(angle), angle)
    out = head.clone()
    out[:, first], out[:, second] = z.real, z.imag
    return out


def _exact_held(x):
    """What x [T, D] becomes in the cache."""
    step = x.abs().max(1, keepdim=True).values / 127
    codes = torch.round(x / torch.where(step == 0, torch.ones_like(step), step))
    return codes.clamp(-127, 127) * step


def exact(case, seed):
    s = prepare(case, seed)
    new, total = lengths(case)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    group = Hq // Hk
    out, at = {}, 0
    if case["op"] == "write":
        T = s["rows"]
        place = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, total)])
        where = place.repeat(max(case["axes"], 1), 1) if s["pos"] is None else s["pos"]
        axis = [0] * (case["rot"] // 2) if s["axis"] is None else s["axis"].tolist()
        angle = torch.stack([where[a].double() * f for a, f in zip(axis, s["inv_freq"].tolist())], 1)
        y = s["y"].double()
        heads = [y[:, h * D:(h + 1) * D] for h in range(Hq + 2 * Hk)]
        q = torch.cat([_exact_turn(h, angle, case["pairs"]) for h in heads[:Hq]], 1)
        k = torch.stack([_exact_held(_exact_turn(h, angle, case["pairs"])) for h in heads[Hq:Hq + Hk]], 1)
        v = torch.stack([_exact_held(h) for h in heads[Hq + Hk:]], 1)
        k[place < 0] = 0
        v[place < 0] = 0
        return {"q": q, "k": k.view(T, Hk, D), "v": v.view(T, Hk, D)}
    if case["op"] == "read":
        both = [_sequence(s, b, t) for b, t in enumerate(total)]
        return {"k": torch.cat([k.transpose(0, 1) for k, _ in both]), "v": torch.cat([v.transpose(0, 1) for _, v in both])}
    o = torch.zeros((s["rows"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], Hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b, (n, t) in enumerate(zip(new, total)):
        q = s["q"][at:at + n].double().view(n, Hq, D)
        if t > 0:
            k, v = _sequence(s, b, t)
            for h in range(Hq):
                for i in range(0, n, 1024):
                    last = torch.arange(t - n + i, t - n + min(i + 1024, n), device="cuda")
                    most = max(int(last[-1]) + 1, 1)
                    x = (q[i:i + 1024, h] @ k[h // group, :most].T) / math.sqrt(D)
                    x = x.masked_fill(torch.arange(most, device="cuda") > last[:, None], float("-inf"))
                    z = torch.logsumexp(x, 1)
                    lse[at + i:at + i + len(last), h] = z
                    w = torch.exp(x - torch.where(last >= 0, z, torch.zeros_like(z))[:, None])
                    o[at + i:at + i + len(last), h] = w @ v[h // group, :most]
        at += n
    out["o"] = o.view(s["rows"], -1)
    if case["lse"]:
        out["lse"] = lse
    return out
