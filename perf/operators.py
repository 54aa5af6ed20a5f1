"""The 8-bit operators as their users call them: cases, plain forms and 64-bit values.

  norm     coda_add_rmsnorm_q8: the residual's addition and the RMS norm with INT8 codes and one
           scale per token, then the codes as the values they stand for (coda_dequant_q8)
  ckpt     coda_quant_q8 and coda_dequant_q8: a tensor saved in 8 bits (a scale per token, or per
           row and 128 columns) and loaded again
  product  coda_matmul_q8: INT8 matrix product with a scale per token and per channel
  bwd      coda_bwd_swiglu_dgrad_q8: the SwiGLU backward with the RMSNorm-branch data gradient from
           an 8-bit checkpoint of the pre-activation, and the gated activation recomputed from it

`run` calls the framework's entry points where `own` is set, and computes the plain form in
elementary torch operations in 32 bits otherwise; `exact` computes the definition in 64 bits.
"""

import math

import torch

own = False

BLOCK = 128  # columns per scale of a checkpoint
EPS = 1e-5


def listed():
    return [
        # one token of a 7B-class model between two projections while decoding
        {"name": "norm_token", "op": "norm", "M": 1, "d": 4096, "z": True},
        # a ragged batch without a residual (the first norm of a stack), odd sizes
        {"name": "norm_ragged", "op": "norm", "M": 997, "d": 5000, "z": False},
        # a prompt of 8192 tokens at a 70B-class width
        {"name": "norm_prefill", "op": "norm", "M": 8192, "d": 8192, "z": True},
        # the gated activation of a decoding batch, one scale per token, for the down projection
        {"name": "ckpt_rows", "op": "ckpt", "M": 32, "n": 14336, "block": 0},
        # a residual stream of odd sizes saved for the backward, last block ragged
        {"name": "ckpt_ragged", "op": "ckpt", "M": 1500, "n": 11000, "block": BLOCK},
        # the SwiGLU pre-activation of the llama7b training step, saved for the backward
        {"name": "ckpt_llama7b", "op": "ckpt", "M": 8192, "n": 28672, "block": BLOCK},
        # gate and up projection of one token: the weights' bytes are the whole cost
        {"name": "product_token", "op": "product", "M": 1, "K": 4096, "N": 28672, "z": False},
        # output projection of a decoding batch onto its residual stream
        {"name": "product_batch", "op": "product", "M": 24, "K": 4096, "N": 4096, "z": True},
        # a chunk of a prompt, odd number of tokens
        {"name": "product_chunk", "op": "product", "M": 333, "K": 4096, "N": 14336, "z": False},
        # gate and up projection of the llama7b shape, 8192 tokens
        {"name": "product_prefill", "op": "product", "M": 8192, "K": 4096, "N": 28672, "z": False},
        # a short ragged batch: latency and partial tiles
        {"name": "bwd_short", "op": "bwd", "M": 77, "d": 264, "N1": 1376, "Dout": 520},
        # the llama7b training step
        {"name": "bwd_llama7b", "op": "bwd", "M": 8192, "d": 4096, "N1": 28672, "Dout": 4096},
    ]


def _spread(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(("norm", "ckpt", "product", "product", "bwd"))
    M = _spread(rng, 1, 8192)
    if op == "norm":
        return {"op": op, "M": M, "d": _spread(rng, 64, 8192, 8), "z": rng.random() < 0.7}
    if op == "ckpt":
        return {"op": op, "M": M, "n": _spread(rng, 64, 28672, 8), "block": rng.choice((0, BLOCK))}
    if op == "product":
        return {"op": op, "M": M, "K": _spread(rng, 64, 8192, 16), "N": _spread(rng, 64, 14336, 16),
                "z": rng.random() < 0.5}
    d = _spread(rng, 64, 4096, 8)
    return {"op": op, "M": M, "d": d, "N1": _spread(rng, 128, 28672, 32),
            "Dout": d if rng.random() < 0.7 else _spread(rng, 64, 4096, 8)}


# --------------------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda")
    return t.normal_(mean, std, generator=gen)


def _codes(gen, shape):
    """Codes of a quantised bell-shaped tensor: most small, the largest at the range's end."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    rows = max(1, (1 << 26) // shape[1])
    for i in range(0, shape[0], rows):
        part = out[i:i + rows]
        part.copy_(_normal(gen, part.shape, 32.0).round_().clamp_(-127, 127))
    return out


def _activation(gen, M, n):
    """bf16 activations with a few loud channels; the last of many rows is padding (zeros)."""
    t = _normal(gen, (M, n))
    t[:, torch.randint(0, n, (max(1, n // 512),), device="cuda", generator=gen)] *= 20.0
    if M >= 8:
        t[M - 1] = 0.0
    return t.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    bf = torch.bfloat16
    s = dict(case)
    M = case["M"]
    if case["op"] == "norm":
        s["x"] = _activation(gen, M, case["d"])
        s["res"] = _activation(gen, M, case["d"]) if case["z"] else None
        s["gamma"] = _normal(gen, (case["d"],), 0.3, 1.0).to(bf)
    elif case["op"] == "ckpt":
        s["x"] = _activation(gen, M, case["n"])
    elif case["op"] == "product":
        K, N = case["K"], case["N"]
        s["a_q"], s["W_q"] = _codes(gen, (M, K)), _codes(gen, (K, N))
        s["a_s"] = torch.rand((M,), device="cuda", generator=gen) * 0.03 + 0.005
        s["w_s"] = torch.rand((N,), device="cuda", generator=gen) * (0.05 / math.sqrt(K)) + 0.01 / math.sqrt(K)
        if M >= 8:  # a padded token
            s["a_q"][M - 1] = 0
            s["a_s"][M - 1] = 0.0
        s["res"] = _normal(gen, (M, N)).to(bf) if case["z"] else None
    else:
        d, N1, Dout = case["d"], case["N1"], case["Dout"]
        s["dout"] = _normal(gen, (M, Dout), 0.1).to(bf)
        s["W2"] = _normal(gen, (N1 // 2, Dout), (2.0 / N1) ** 0.5).to(bf)
        s["W1"] = _normal(gen, (d, N1), d ** -0.5).to(bf)
        s["y_q"] = _codes(gen, (M, N1))
        s["y_s"] = torch.rand((M, -(-N1 // BLOCK)), device="cuda", generator=gen) * 0.02 + 0.015
        h = _normal(gen, (M, d), 1.5)
        s["h"], s["r"] = h.to(bf), (h.square().mean(1) + EPS).rsqrt()
        s["gamma"] = _normal(gen, (d,), 0.3, 1.0).to(bf)
    return s


# --------------------------------------------------------------------------- one pass
def _plain_codes(u, block):
    """The values that u's INT8 codes stand for and their scales: amax / 127 of each row
    (block 0) or of each `block` columns of a row; a scale of zero for zeros alone."""
    M, n = u.shape
    width = block or n
    cut = torch.nn.functional.pad(u, (0, -n % width)).view(M, -1, width)
    amax = cut.abs().amax(2, keepdim=True)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    scale = amax / 127.0
    return (torch.round(cut * inv) * scale).view(M, -1)[:, :n], scale.squeeze(2)


def _wide(scales, n):
    """Scales per 128 columns, one for each of n columns."""
    return scales.repeat_interleave(BLOCK, 1)[:, :n]


def _plain(s):
    bf = torch.bfloat16
    if s["op"] == "norm":
        h = s["x"].float()
        if s["res"] is not None:
            h = h + s["res"].float()
        r = (h.square().mean(1, keepdim=True) + EPS).rsqrt()
        values, scale = _plain_codes(r * h * s["gamma"].float(), 0)
        out = {"values": values.to(bf), "scale": scale[:, 0]}
        return dict(out, h=h.to(bf)) if s["res"] is not None else out
    if s["op"] == "ckpt":
        values, scale = _plain_codes(s["x"].float(), s["block"])
        return {"values": values.to(bf), "scale": scale if s["block"] else scale[:, 0]}
    if s["op"] == "product":
        y = (s["a_q"].float() @ s["W_q"].float()) * s["a_s"][:, None] * s["w_s"]
        return {"y": (y if s["res"] is None else y + s["res"].float()).to(bf)}
    n1, d = s["N1"], s["d"]
    da = s["dout"].float() @ s["W2"].float().t()
    y = s["y_q"].float() * _wide(s["y_s"], n1)
    g, u = y[:, :n1 // 2], y[:, n1 // 2:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    dy = torch.cat((da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig), 1)
    stat = (dy * y).sum(1)
    r = s["r"][:, None]
    dh = r * s["gamma"].float() * (dy @ s["W1"].float().t()) - r * r * stat[:, None] / d * s["h"].float()
    return {"dy": dy.to(bf), "s": stat, "dh": dh.to(bf), "a": (g * sig * u).to(bf)}


def run(s):
    if not own:
        return _plain(s)
    from gemm_epilogue_fusion_gemm0_gb300 import binding as B

    if s["op"] == "norm":
        h, q, scale = B.coda_add_rmsnorm_q8(s["x"], s["gamma"], EPS, z=s["res"])
        out = {"values": B.coda_dequant_q8(q, scale), "scale": scale}
        return dict(out, h=h) if s["res"] is not None else out
    if s["op"] == "ckpt":
        q, scale = B.coda_quant_q8(s["x"], block=s["block"])
        return {"values": B.coda_dequant_q8(q, scale, block=s["block"]), "scale": scale}
    if s["op"] == "product":
        return {"y": B.coda_matmul_q8(s["a_q"], s["a_s"], s["W_q"], s["w_s"], z=s["res"])}
    dy, stat, dh, a = B.coda_bwd_swiglu_dgrad_q8(s["dout"], s["W2"], s["y_q"], s["y_s"], s["W1"],
                                                 s["h"], s["r"], s["gamma"], want_a=True)
    return {"dy": dy, "s": stat, "dh": dh, "a": a}


# --------------------------------------------------------------------------- work
def work(case):
    M = case["M"]
    if case["op"] == "norm":  # x, the residual, gamma; h, the values, the scales
        d = case["d"]
        return {"bytes": 2 * M * d * (4 if case["z"] else 2) + 2 * d + 4 * M,
                "flops": (9 if case["z"] else 8) * M * d}
    if case["op"] == "ckpt":
        n = case["n"]
        scales = M * (-(-n // case["block"]) if case["block"] else 1)
        return {"bytes": 4 * M * n + 4 * scales, "flops": 4 * M * n}
    if case["op"] == "product":
        K, N = case["K"], case["N"]
        return {"bytes": M * K + K * N + 4 * (M + N) + 2 * M * N * (2 if case["z"] else 1),
                "flops": 2 * M * K * N}
    d, N1, Dout = case["d"], case["N1"], case["Dout"]
    blocks = -(-N1 // BLOCK)
    return {"bytes": 2 * (M * Dout + N1 // 2 * Dout + d * N1 + M * d + d) + M * N1 + 4 * M * blocks
            + 4 * M + 2 * (M * N1 + M * N1 // 2 + M * d) + 4 * M,
            "flops": 2 * M * Dout * (N1 // 2) + 2 * M * N1 * d}


# --------------------------------------------------------------------------- 64 bits
def _exact_quantised(v, width):
    M, n = v.shape
    values, scales = torch.empty_like(v), []
    for at in range(0, n, width):
        part = v[:, at:at + width]
        step = part.abs().max(1).values / 127
        scales.append(step)
        safe = torch.where(step > 0, step, torch.ones_like(step))[:, None]
        values[:, at:at + width] = torch.clamp(torch.round(part / safe), -127, 127) * step[:, None]
    return values, torch.stack(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    f = lambda name: s[name].double()  # noqa: E731
    if case["op"] == "norm":
        h = f("x") if s["res"] is None else f("x") + f("res")
        norm = torch.sqrt(torch.mean(h * h, 1) + EPS)
        values, scales = _exact_quantised(h / norm[:, None] * f("gamma"), case["d"])
        out = {"values": values, "scale": scales[:, 0]}
        return dict(out, h=h) if s["res"] is not None else out
    if case["op"] == "ckpt":
        values, scales = _exact_quantised(f("x"), case["block"] or case["n"])
        return {"values": values, "scale": scales if case["block"] else scales[:, 0]}
    if case["op"] == "product":
        y = torch.matmul(f("a_q") * f("a_s")[:, None], f("W_q") * f("w_s")[None, :])
        return {"y": y if s["res"] is None else f("res") + y}
    half, d = case["N1"] // 2, case["d"]
    y = f("y_q")
    for b in range(s["y_s"].shape[1]):
        y[:, b * BLOCK:(b + 1) * BLOCK] *= f("y_s")[:, b:b + 1]
    gate, up = y[:, :half], y[:, half:]
    da = torch.matmul(f("dout"), f("W2").T)
    sg = torch.sigmoid(gate)
    silu = gate * sg
    dg = da * up * (sg + silu * (1 - sg))
    du = da * silu
    stat = (dg * gate).sum(1) + (du * up).sum(1)
    W1 = f("W1")
    t = torch.matmul(dg, W1[:, :half].T) + torch.matmul(du, W1[:, half:].T)
    r = f("r")[:, None]
    dh = r * (f("gamma") * t) - r ** 2 * (stat / d)[:, None] * f("h")
    return {"dy": torch.cat((dg, du), 1), "s": stat, "dh": dh, "a": silu * up}
