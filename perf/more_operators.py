"""Cases of the operators that complete a decoder block around the quantized products and the 4-bit cache.

Four operators, in the order in which a block meets them:

  norm      the norms after and before a block, fused with the gate and the
            residual stream between them
  quantize  rows in microscaled blocks: 4-bit (E2M1) or 8-bit (E4M3) floats, 32
            sharing a power of two
  product   y = residual + act(W x + bias), or residual + act(gate) * up, W in
            E2M1 blocks, x in E2M1 or E4M3 blocks or quantised on the way
  rotary    queries and keys rotated by position (one axis, or time, height and
            width), keys and values appended to the 4-bit paged cache

``run`` computes them in plain torch operations, or, where ``own`` is set,
calls the package.
"""

import math

import torch

own = False

DEV = "cuda"
_TYPE = {"fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def _quantize(name, T, K, dtype, fmt, clip):
    return {"name": name, "op": "quantize", "T": T, "K": K, "dtype": dtype, "fmt": fmt, "clip": clip}


def _product(name, T, M, K, x, fmt, act, gated, bias, residual, out):
    """x: "rows" (FP16, quantised by the call) or "blocks" (quantised before it, by a norm say)."""
    return {"name": name, "op": "product", "T": T, "M": M, "K": K, "x": x, "fmt": fmt, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "out": out}


def _norm(name, T, N, kind, y, stream, post, gate, scale, out):
    """stream: type of the residual stream; gate: "none", "channel" [N] or "row" [T, N]; out: a type or a block format."""
    return {"name": name, "op": "norm", "T": T, "N": N, "kind": kind, "y": y, "stream": stream, "post": post,
            "gate": gate, "scale": scale, "out": out}


def _rotary(name, seqs, past, new, q_heads, heads, dim, rot, style, axes, base, group, page):
    return {"name": name, "op": "rotary", "seqs": seqs, "past": past, "new": new, "q_heads": q_heads, "heads": heads,
            "dim": dim, "rot": rot, "style": style, "axes": axes, "base": base, "group": group, "page": page}


def listed():
    return [
        # one decoding step of sixteen sequences before the 70B-shaped MLP
        _quantize("quantize_step_16", 16, 8192, "fp16", "e2m1", False),
        # a long prompt's activations before the 7B MLP's down projection, kept in 8 bits
        _quantize("quantize_prompt", 8190, 11008, "fp32", "e4m3", True),
        # the 7B block's attention output projection for one token, added to the residual stream
        _product("product_o_1", 1, 4096, 4096, "rows", "e4m3", "none", False, False, True, "fp16"),
        # the 70B-shaped MLP projection for one token, biased and activated
        _product("product_mlp70b_1", 1, 28672, 8192, "blocks", "e2m1", "gelu_tanh", False, True, False, "fp32"),
        # the 7B block's gate and up projections as one gated product for sixteen sequences
        _product("product_gate_up_16", 16, 22016, 4096, "rows", "e4m3", "silu", True, False, False, "fp16"),
        # the 7B block's down projection for a few sequences with drafted tokens
        _product("product_down_61", 61, 4096, 11008, "blocks", "e2m1", "none", False, False, True, "fp16"),
        # a prompt through the 7B block's gate and up projections
        _product("product_gate_up_2043", 2043, 22016, 4096, "blocks", "e2m1", "silu", True, False, False, "fp16"),
        # many prompts together through the 70B-shaped MLP projection
        _product("product_mlp70b_8192", 8192, 28672, 8192, "rows", "e2m1", "none", False, False, False, "fp16"),
        # one token between two blocks of the 70B shape, the stream in FP16
        _norm("norm_step_1", 1, 8192, "rms", "fp16", "fp16", True, "none", 1.0, "fp16"),
        # many prompts between two blocks, each row with a gate of its own, straight into blocks for the next product
        _norm("norm_prompt_8190", 8190, 4096, "layer", "fp16", "fp32", False, "row", 1.0, "e4m3"),
        # one decoding step of sixteen sequences of the 7B block's heads
        _rotary("rotary_step_16", 16, 1500, 1, 32, 32, 128, 128, "halves", 1, 10000.0, 32, 64),
        # a long video's tokens of the 70B-shaped heads, positions in time, height and width
        _rotary("rotary_video", 3, 37, 10007, 64, 8, 128, 128, "halves", 3, 1000000.0, 64, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "norm", "rotary"])
    if op == "quantize":
        K = 32 * _log(rng, 1, 896)
        c = _quantize("", min(_log(rng, 1, 16384), 8190 * 11008 // K), K, rng.choice(["fp16", "fp32"]),
                      rng.choice(["e2m1", "e4m3"]), rng.random() < 0.5)
    elif op == "product":
        K = 32 * _log(rng, 2, 350)
        M = 2 * _log(rng, 8, 14336)
        T = max(1, min(_log(rng, 1, 8192), 8192 * 28672 * 8192 // (2 * M * K)))
        c = _product("", T, M, K, rng.choice(["rows", "blocks"]), rng.choice(["e2m1", "e4m3"]),
                     rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.4,
                     rng.random() < 0.5, rng.random() < 0.5, rng.choice(["fp16", "fp32"]))
    elif op == "norm":
        N = 32 * _log(rng, 2, 512)
        # E2M1's steps are so far apart that one value next to a border, which 32 bits send either way, decides a comparison
        out = rng.choice(["fp16", "fp32", "e4m3"])
        c = _norm("", min(_log(rng, 1, 16384), 8190 * 4096 // N), N, rng.choice(["rms", "layer"]),
                  rng.choice(["fp16", "fp32"]), rng.choice(["fp16", "fp32"]), rng.random() < 0.5,
                  rng.choice(["none", "channel", "row"]), rng.choice([1.0, 0.5]), out)
    else:
        dim = rng.choice([64, 128, 256])
        heads = rng.choice([1, 2, 4, 8, 16, 32])
        per = rng.choice([1, 2, 4, 7, 8])
        seqs = rng.choice([1, 2, 5, 8, 16])
        new = _log(rng, 1, 3 * 10007 * 80 * 128 // (seqs * heads * (per + 2) * dim))
        c = _rotary("", seqs, _log(rng, 1, 100000) - 1, new, heads * per, heads, dim,
                    rng.choice([dim, dim, dim // 2, dim // 4]), rng.choice(["halves", "neighbours"]),
                    rng.choice([1, 1, 2, 3]), rng.choice([10000.0, 500000.0]),
                    rng.choice([g for g in (32, 64, 128) if g <= dim]), rng.choice([16, 32, 64, 128, 256]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
_BITS = {"e2m1": 4.25, "e4m3": 8.25}  # with the block's power of two


def _blocks_bytes(n, fmt):
    return int(n * _BITS[fmt]) // 8


def work(case):
    op = case["op"]
    if op == "quantize":
        # values in, blocks out, the same blocks in, the values that they stand for out
        n = case["T"] * case["K"]
        return {"bytes": 2 * n * _SIZE[case["dtype"]] + 2 * _blocks_bytes(n, case["fmt"]), "flops": 4 * n}
    if op == "product":
        T, M, K = case["T"], case["M"], case["K"]
        mo = M // 2 if case["gated"] else M
        b = _blocks_bytes(M * K, "e2m1") + _SIZE[case["out"]] * T * mo
        b += 2 * T * K if case["x"] == "rows" else _blocks_bytes(T * K, case["fmt"])
        b += (2 * M if case["bias"] else 0) + (2 * T * mo if case["residual"] else 0)
        return {"bytes": b, "flops": 2 * T * M * K}
    if op == "norm":
        n, N = case["T"] * case["N"], case["N"]
        b = n * (_SIZE[case["y"]] + 2 * _SIZE[case["stream"]]) + 2 * N * (1 + 2 * case["post"] + (case["kind"] == "layer"))
        b += {"none": 0, "channel": 2 * N, "row": 2 * n}[case["gate"]]
        # blocks are returned as the values that they stand for, so they are read again and those written
        b += n * _SIZE[case["out"]] if case["out"] in _SIZE else 2 * _blocks_bytes(n, case["out"]) + 2 * n
        return {"bytes": b, "flops": 12 * n}
    t, H, D = case["seqs"] * case["new"], case["heads"], case["dim"]
    codes = t * H * 2 * (D // 2 + 4 * (D // case["group"]))
    # queries in and out, keys and values in, codes out, the same codes in, keys and values out
    b = 2 * t * D * (2 * case["q_heads"] + 2 * H + 2 * H) + 2 * codes
    return {"bytes": b + (4 * t * case["axes"] if case["axes"] > 1 else 0), "flops": t * D * (3 * case["q_heads"] + 14 * H)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * seed + sum(ord(c) * (i + 1) for i, c in enumerate(repr(sorted(
        (k, v) for k, v in case.items() if k != "name")))) % 1000003)
    return g


def _randn(g, shape, dtype="fp32"):
    return torch.randn(shape, generator=g, device=DEV).to(_TYPE[dtype])


def _activations(g, T, K, dtype):
    """Rows of a layer's activations: normal, every channel with a size of its own, a few of them large."""
    size = torch.exp(0.5 * torch.randn(K, generator=g, device=DEV))
    size = torch.where(torch.rand(K, generator=g, device=DEV) < 0.005, 20 * size, size)
    return (torch.randn((T, K), generator=g, device=DEV) * size).to(_TYPE[dtype])


def _weight_blocks(g, M, K):
    """A weight set in E2M1 blocks: codes uint8 [M, K / 2], the lower nibble first, and exponents uint8 [M, K / 32]."""
    codes = torch.randint(0, 256, (M, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    # blocks of weights of about 0.02: powers of two from 2^-9 to 2^-6
    return codes, torch.randint(127 - 9, 127 - 5, (M, K // 32), generator=g, device=DEV, dtype=torch.uint8)


def _product_inputs(case, seed):
    g = _gen(case, seed)
    T, M, K = case["T"], case["M"], case["K"]
    mo = M // 2 if case["gated"] else M
    codes, exps = _weight_blocks(g, M, K)
    x = _activations(g, T, K, "fp16")
    bias = _randn(g, M, "fp16") if case["bias"] else None
    residual = _randn(g, (T, mo), "fp16") if case["residual"] else None
    return codes, exps, x, bias, residual


def _norm_inputs(case, seed):
    g = _gen(case, seed)
    T, N = case["T"], case["N"]
    st = {"y": _activations(g, T, N, case["y"]), "h": 3 * _activations(g, T, N, case["stream"]) + 0.25}
    one = lambda: (1 + 0.2 * _randn(g, N)).half()  # noqa: E731
    st["post"] = one() if case["post"] else None
    st["pre"] = one()
    st["post_bias"] = (0.1 * _randn(g, N)).half() if case["post"] and case["kind"] == "layer" else None
    st["pre_bias"] = (0.1 * _randn(g, N)).half() if case["kind"] == "layer" else None
    gate = {"none": None, "channel": (N,), "row": (T, N)}[case["gate"]]
    st["gate"] = None if gate is None else _randn(g, gate, "fp16")
    return st


def _rotary_inputs(case, seed):
    g = _gen(case, seed)
    S, n, D, page = case["seqs"], case["new"], case["dim"], case["page"]
    t, length = S * n, case["past"] + n
    st = {"q": 2 * _randn(g, (t, case["q_heads"], D), "fp16")}
    # keys sit around an offset per channel, values around zero
    st["k"] = (_randn(g, (t, case["heads"], D)) + 2 * _randn(g, (case["heads"], D))).half()
    st["v"] = _randn(g, (t, case["heads"], D), "fp16")
    need = -(-length // page)
    # a pool with a few spare pages, in shuffled order
    st["total"] = S * need + 3
    st["pages"] = torch.randperm(st["total"], generator=g, device=DEV)[:S * need].to(torch.int32).view(S, need)
    pairs = case["rot"] // 2
    st["freqs"] = case["base"] ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
    st["positions"] = st["pair_axis"] = None
    if case["axes"] > 1:
        # frames of 24 x 40 tokens behind what the sequence holds already; the pairs are dealt out in sections
        i = torch.arange(n, device=DEV)
        p = torch.stack([i // 960, i // 40 % 24, i % 40])[:case["axes"]] + case["past"]
        st["positions"] = p.to(torch.int32).repeat(1, S)
        st["pair_axis"] = torch.arange(pairs, device=DEV) * case["axes"] // pairs
    st["length"] = length
    return st


def prepare(case, seed):
    if case["op"] == "quantize":
        return {"case": case, "x": _activations(_gen(case, seed), case["T"], case["K"], case["dtype"])}
    if case["op"] == "norm":
        return {"case": case, **_norm_inputs(case, seed)}
    if case["op"] == "product":
        codes, exps, x, bias, residual = _product_inputs(case, seed)
        st = {"case": case, "x": x, "bias": bias, "residual": residual}
        if own:
            from dense_sparse_bit_amd import qmx
            st["plan"] = qmx.QMx(qmx.MxRows.pack(codes, exps))
            if case["x"] == "blocks":
                st["x"] = qmx.quantize(x, case["fmt"])
        else:
            st["codes"], st["exps"] = codes, exps
            if case["x"] == "blocks":
                st["x"] = _plain_quantize(x, case["fmt"], False)
        return st
    st = {"case": case, **_rotary_inputs(case, seed)}
    if own:
        from dense_sparse_bit_amd import qcache, qrotary
        S, n = case["seqs"], case["new"]
        st["cache"] = qcache.QCache(st["total"], case["heads"], case["dim"], page_size=case["page"], group=case["group"])
        st["rotary"] = qrotary.Rotary(st["freqs"], style=case["style"], pair_axis=st["pair_axis"])
        st["lens"] = torch.full((S,), st["length"], dtype=torch.int32, device=DEV)
        st["q_start"] = None if n == 1 else torch.arange(S + 1, dtype=torch.int32, device=DEV) * n
    else:
        p = torch.arange(st["length"] - case["new"], st["length"], device=DEV)
        st["slots"] = (st["pages"].long()[:, p // case["page"]] * case["page"] + p % case["page"]).reshape(-1)
        st["pool"] = [_pool(st["total"] * case["page"], case) for _ in range(2)]
        st["at"] = p.repeat(case["seqs"])
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_quantize(x, fmt, clip):
    """(elements, power of two) of blocks of 32, fp32 [T, K / 32, 32] and [T, K / 32, 1].

    The power of two is the smallest that reaches the block's largest value or, clipping, the largest value's own less
    the element's; elements are rounded to nearest, ties to even, and stop at the format's largest.
    """
    b = x.float().view(x.shape[0], x.shape[1] // 32, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    if fmt == "e2m1":  # largest 6 = 0.75 2^3
        e = e - 3 + (0 if clip else (m > 0.75).int())
    else:  # largest 448 = 0.875 2^9
        e = e - 9 + (0 if clip else (m > 0.875).int())
    step = torch.ldexp(torch.ones_like(top), e.clamp(min=-126))
    v = b / step
    a = v.abs()
    if fmt == "e2m1":
        unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        largest = 6.0
    else:
        unit = torch.ldexp(torch.ones_like(a), (torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
        largest = 448.0
    return torch.copysign((torch.round(a / unit) * unit).clamp(max=largest), v), step


def _plain_weights(codes, exps):
    """fp32 [M, K] of E2M1 blocks."""
    q = torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], exps.shape[1], 32)
    m = (q & 7).float()
    # 0, 0.5, 1, 1.5, 2, 3, 4, 6
    mag = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    step = torch.ldexp(torch.ones_like(exps, dtype=torch.float32), exps.int() - 127)
    return (torch.where(q > 7, -mag, mag) * step[:, :, None]).view(codes.shape[0], -1)


def _plain_act(t, act):
    if act == "relu":
        return torch.where(t > 0, t, torch.zeros_like(t))
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return 0.5 * t * torch.erfc(t * -0.7071067811865476)
    if act == "gelu_tanh":
        return t / (1 + torch.exp(-1.5957691216057308 * (t + 0.044715 * t * t * t)))
    return t


def _plain_product(st):
    case = st["case"]
    el, step = _plain_quantize(st["x"], case["fmt"], False) if case["x"] == "rows" else st["x"]
    t = (el * step).view(case["T"], case["K"]) @ _plain_weights(st["codes"], st["exps"]).t()
    if st["bias"] is not None:
        t = t + st["bias"].float()
    if case["gated"]:
        t = _plain_act(t[:, 0::2], case["act"]) * t[:, 1::2]
    else:
        t = _plain_act(t, case["act"])
    if st["residual"] is not None:
        t = t + st["residual"].float()
    return t.to(_TYPE[case["out"]])


def _plain_unit(x, kind, weight, bias):
    if kind == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(dim=1, keepdim=True) + 1e-6) * weight.float()
    return x if bias is None else x + bias.float()


def _plain_norm(st):
    case = st["case"]
    b = st["y"].float()
    if st["post"] is not None:
        b = _plain_unit(b, case["kind"], st["post"], st["post_bias"])
    if st["gate"] is not None:
        b = st["gate"].float() * b
    h = case["scale"] * st["h"].float() + b
    out = _plain_unit(h, case["kind"], st["pre"], st["pre_bias"])
    if case["out"] in _TYPE:
        out = out.to(_TYPE[case["out"]])
    else:
        el, step = _plain_quantize(out, case["out"], False)
        out = (el * step).view(out.shape).half()
    return h.to(_TYPE[case["stream"]]), out


def _pool(slots, case):
    """Plain 4-bit storage of keys or values: codes, step and lowest value per group."""
    H, D, G = case["heads"], case["dim"], case["group"]
    return {"q": torch.zeros((slots, H, D // 2), dtype=torch.uint8, device=DEV),
            "s": torch.zeros((slots, H, D // G), dtype=torch.float16, device=DEV),
            "lo": torch.zeros((slots, H, D // G), dtype=torch.float16, device=DEV)}


def _plain_held(pool, slots, val, G):
    """Writes FP16 rows into the pool, and reads them back."""
    t, H, D = val.shape
    x = val.float().view(t, H, D // G, G)
    lo = x.amin(dim=3)
    s = ((x.amax(dim=3) - lo) / 15).half()
    q = torch.round((x - lo[..., None]) / s.float()[..., None])
    q = torch.where(s[..., None] > 0, q, torch.zeros_like(q)).clamp(0, 15).to(torch.uint8).view(t, H, D)
    pool["q"][slots] = q[..., 0::2] | (q[..., 1::2] << 4)
    pool["s"][slots] = s
    pool["lo"][slots] = lo.half()
    p = pool["q"][slots]
    q = torch.stack([p & 15, p >> 4], dim=3).view(t, H, D // G, G).float()
    return (q * pool["s"][slots].float()[..., None] + pool["lo"][slots].float()[..., None]).view(t, H, D).half()


def _plain_turned(x, cos, sin, rot, style):
    """x [t, heads, D] with its first rot dimensions turned, in 64 bits: keys next to a border go either way."""
    y = x.double()
    if style == "halves":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    c, s = cos[:, None], sin[:, None]
    pair = (a * c - b * s, b * c + a * s)
    turned = torch.cat(pair, dim=-1) if style == "halves" else torch.stack(pair, dim=-1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], dim=-1).half()


def _plain_rotary(st):
    case = st["case"]
    if st["positions"] is None:
        at = st["at"][:, None].double()
    else:
        at = st["positions"][st["pair_axis"]].t().double()
    angle = at * st["freqs"]
    cos, sin = torch.cos(angle), torch.sin(angle)
    q = _plain_turned(st["q"], cos, sin, case["rot"], case["style"])
    k = _plain_turned(st["k"], cos, sin, case["rot"], case["style"])
    return (q, _plain_held(st["pool"][0], st["slots"], k, case["group"]),
            _plain_held(st["pool"][1], st["slots"], st["v"], case["group"]))


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "quantize":
            el, step = _plain_quantize(state["x"], case["fmt"], case["clip"])
            return (el * step).view(state["x"].shape).to(_TYPE[case["dtype"]])
        return {"product": _plain_product, "norm": _plain_norm, "rotary": _plain_rotary}[op](state)
    from dense_sparse_bit_amd import qmx, qnorm
    if op == "quantize":
        return qmx.quantize(state["x"], case["fmt"], clip=case["clip"]).values(_TYPE[case["dtype"]])
    if op == "product":
        return state["plan"].run(state["x"], x_fmt=case["fmt"], bias=state["bias"], act=case["act"], gated=case["gated"],
                                 residual=state["residual"], dtype=_TYPE[case["out"]])
    if op == "norm":
        h, out = qnorm.norm(state["y"], state["h"], post=state["post"], post_bias=state["post_bias"], gate=state["gate"],
                            scale=case["scale"], pre=state["pre"], pre_bias=state["pre_bias"], kind=case["kind"],
                            eps=1e-6, out_type=case["out"])
        return h, out if case["out"] in _TYPE else out.values(torch.float16)
    q = state["rotary"].write(state["cache"], state["q"], state["k"], state["v"], state["lens"], state["pages"],
                              state["q_start"], positions=state["positions"])
    k, v = state["cache"].read(state["lens"], state["pages"], state["q_start"], n_tok=state["k"].shape[0])
    return q, k, v


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def _exact_grid(fmt):
    """The format's values from 0 up, in 64 bits."""
    if fmt == "e2m1":
        v = [(1 + m / 2) * 2.0 ** (e - 1) if e else m / 2 for e in range(4) for m in range(2)]
    else:
        v = [(1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9 for e in range(16) for m in range(8)][:-1]
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_blocks(x, fmt, clip):
    """The values that x's blocks stand for: each the nearest of the grid, an even index where two are as near."""
    grid = _exact_grid(fmt)
    b = x.double().view(-1, 32)
    top = b.abs().max(dim=1, keepdim=True).values
    if clip:  # the largest value's binade lands on the grid's last
        step = torch.exp2((torch.floor(torch.log2(top)) - math.floor(math.log2(grid[-1].item()))).clamp(min=-126))
    else:
        step = torch.exp2(torch.ceil(torch.log2(top / grid[-1])).clamp(min=-126))
        # log2 may be off by its last bit next to a border
        step = torch.where(top > grid[-1] * step, 2 * step, step)
        step = torch.where((top <= grid[-1] * step / 2) & (step > 2.0 ** -126), step / 2, step)
    a = b.abs() / step
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    i = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (torch.sign(b) * grid[i] * step).view(x.shape)


def _exact_product(case, seed):
    codes, exps, x, bias, residual = _product_inputs(case, seed)
    M, K = case["M"], case["K"]
    lut = torch.cat([_exact_grid("e2m1"), -_exact_grid("e2m1")])
    xv = _exact_blocks(x, case["fmt"], False)
    mo = M // 2 if case["gated"] else M
    out = torch.empty((case["T"], mo), dtype=torch.float64, device=DEV)
    rows = 4096
    for r in range(0, M, rows):
        c = codes[r:r + rows]
        w = torch.empty((c.shape[0], K), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = lut[(c % 16).long()], lut[(c // 16).long()]
        w *= torch.exp2(exps[r:r + rows].double() - 127).repeat_interleave(32, dim=1)
        t = xv @ w.t()
        if bias is not None:
            t += bias[r:r + rows].double()
        u = t[:, ::2] if case["gated"] else t
        if case["act"] == "relu":
            u = torch.clamp(u, min=0)
        elif case["act"] == "silu":
            u = u * torch.sigmoid(u)
        elif case["act"] == "gelu":
            u = u * torch.special.ndtr(u)
        elif case["act"] == "gelu_tanh":
            u = u * torch.sigmoid(math.sqrt(8 / math.pi) * (u + 0.044715 * u ** 3))
        if case["gated"]:
            out[:, r // 2:r // 2 + u.shape[1]] = u * t[:, 1::2]
        else:
            out[:, r:r + u.shape[1]] = u
    if residual is not None:
        out += residual.double()
    return out


def _exact_norm(case, seed):
    st = _norm_inputs(case, seed)
    st = {k: None if v is None else v.double() for k, v in st.items()}

    def unit(x, weight, bias):
        mean = x.mean(dim=1, keepdim=True) if case["kind"] == "layer" else 0.0
        r = torch.rsqrt(((x - mean) ** 2).mean(dim=1, keepdim=True) + 1e-6)
        return (x - mean) * r * weight + (0.0 if bias is None else bias)

    b = st["y"] if st["post"] is None else unit(st["y"], st["post"], st["post_bias"])
    h = case["scale"] * st["h"] + (b if st["gate"] is None else st["gate"] * b)
    out = unit(h, st["pre"], st["pre_bias"])
    return h, out if case["out"] in _TYPE else _exact_blocks(out, case["out"], False)


def _exact_held(x, G):
    """lo + s q in 64 bits of FP16 rows x.  The storage is defined with an FP16 step and a quotient of FP32, so those are
    kept."""
    t, H, D = x.shape
    x = x.double().view(t, H, D // G, G)
    lo, hi = x.min(dim=3, keepdim=True).values, x.max(dim=3, keepdim=True).values
    s = ((hi - lo).float() / 15).half()
    q = ((x - lo).float() / s.float()).double().round().clamp(0, 15)
    return (lo + torch.where(s > 0, s.double() * q, torch.zeros_like(q))).view(t, H, D)


def _exact_rotary(case, seed):
    st = _rotary_inputs(case, seed)
    n, rot, pairs = case["new"], case["rot"], case["rot"] // 2
    if st["positions"] is None:
        where = (torch.arange(n, device=DEV) + case["past"]).repeat(case["seqs"])[:, None].expand(-1, pairs)
    else:
        where = torch.stack([st["positions"][int(a)] for a in st["pair_axis"]], dim=1)
    # unit complex numbers
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), where.double() * st["freqs"])[:, None]

    def turned(x):
        y = x.double()
        first = torch.arange(pairs, device=DEV) if case["style"] == "halves" else 2 * torch.arange(pairs, device=DEV)
        second = first + (pairs if case["style"] == "halves" else 1)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    # the cache takes keys in FP16
    return turned(st["q"]), _exact_held(turned(st["k"]).half(), case["group"]), _exact_held(st["v"], case["group"])


def exact(case, seed):
    if case["op"] == "quantize":
        return _exact_blocks(_activations(_gen(case, seed), case["T"], case["K"], case["dtype"]), case["fmt"], case["clip"])
    return {"product": _exact_product, "norm": _exact_norm, "rotary": _exact_rotary}[case["op"]](case, seed)
