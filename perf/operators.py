"""Cases of the decoder-step operators around the quantized products.

Three operators, in the order a decoder block uses them:

  product   y = residual + act(W x + bias), or residual + act(gate) * up with
            the gate and up rows interleaved, W in the dense-and-sparse
            quantized formats (uniform, LUT, BPDQ)
  cache     keys and values quantised to 4 bits as they are written into a
            paged cache, and read back
  attend    a step's queries over that cache, grouped heads, causal at the
            end of each sequence

``run`` computes them in plain torch operations, or, where ``own`` is set,
calls the package.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def _product(name, fmt, bits, M, K, group, density, batch, act, gated, bias, residual, out):
    return {"name": name, "op": "product", "fmt": fmt, "bits": bits, "M": M, "K": K, "group": group,
            "density": density, "batch": batch, "act": act, "gated": gated, "bias": bias, "residual": residual,
            "out": out}


def _cache(name, seqs, past, new, heads, dim, group, page, dtype, out):
    return {"name": name, "op": "cache", "seqs": seqs, "past": past, "new": new, "heads": heads, "dim": dim,
            "group": group, "page": page, "dtype": dtype, "out": out}


def _attend(name, seqs, shortest, longest, new, q_heads, heads, dim, group, page):
    return {"name": name, "op": "attend", "seqs": seqs, "shortest": shortest, "longest": longest, "new": new,
            "q_heads": q_heads, "heads": heads, "dim": dim, "group": group, "page": page}


def listed():
    return [
        # the 7B block's attention output projection for one token, added to the residual stream
        _product("product_o_u3_b1", "uniform", 3, 4096, 4096, 16, 0.005, 1, "none", False, False, True, "fp16"),
        # the 7B block's down projection for sixteen sequences, added to the residual stream
        _product("product_down_u3_b16", "uniform", 3, 4096, 11008, 16, 0.01, 16, "none", False, False, True, "fp16"),
        # the 7B block's gate and up projections as one gated product for sixteen sequences
        _product("product_gate_up_u3_b16", "uniform", 3, 22016, 4096, 16, 0.01, 16, "silu", True, False, False, "fp16"),
        # the 70B-shaped MLP projection for one token, biased and activated
        _product("product_mlp70b_lut4_b1", "lut", 4, 28672, 8192, 0, 0.005, 1, "gelu_tanh", False, True, False, "fp32"),
        # the 7B MLP's up projection in bit planes for eight sequences
        _product("product_mlp7b_bpdq3_b8", "bpdq", 3, 11008, 4096, 64, 0.0045, 8, "relu", False, True, False, "fp16"),
        # one decoding step of sixteen sequences: a token's keys and values each
        _cache("cache_step_16", 16, 1500, 1, 32, 128, 32, 64, "fp16", "fp16"),
        # four prompts written behind a shared prefix and read back rounded for their own attention
        _cache("cache_prompt_4", 4, 37, 2043, 8, 128, 64, 64, "fp32", "fp16"),
        # one long document
        _cache("cache_long", 1, 0, 65536, 8, 128, 32, 128, "fp16", "fp32"),
        # one chat turn of the 7B block's heads, where latency counts
        _attend("attend_short", 1, 181, 181, 1, 32, 32, 128, 32, 64),
        # the 7B block's heads over one long context
        _attend("attend_one_long", 1, 32768, 32768, 1, 32, 32, 128, 32, 64),
        # sixteen ragged sequences of the 70B-shaped heads, two tokens each (one drafted)
        _attend("attend_16_ragged", 16, 333, 8011, 2, 64, 8, 128, 64, 16),
        # sixteen long contexts of the 70B-shaped heads
        _attend("attend_16_long", 16, 32768, 32768, 1, 64, 8, 128, 32, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "cache", "attend"])
    if op == "product":
        fmt, bits = rng.choice([("uniform", 3), ("uniform", 4), ("lut", 3), ("lut", 4), ("bpdq", 3)])
        group = {"uniform": 16, "lut": 0}.get(fmt) if fmt != "bpdq" else rng.choice([32, 64, 128])
        step = max(32, group)
        K = max(step, _log(rng, 256, 11008) // step * step)
        M = min(_log(rng, 512, 28672), 28672 * 8192 // K)
        gated = rng.random() < 0.4
        if gated:
            M -= M % 2
        return {k: v for k, v in _product(
            "", fmt, bits, M, K, group, rng.choice([0.0, 0.0045, 0.01]), rng.choice([1, 8, 16]),
            rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), gated, rng.random() < 0.5,
            rng.random() < 0.5, rng.choice(["fp16", "fp32"])).items() if k != "name"}
    dim = rng.choice([64, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    heads = rng.choice([1, 2, 4, 8, 16, 32])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "cache":
        seqs = rng.choice([1, 2, 5, 8, 16])
        new = _log(rng, 1, 40000000 // (seqs * heads * dim))
        return {k: v for k, v in _cache("", seqs, _log(rng, 1, 2000) - 1, new, heads, dim, group, page,
                                        rng.choice(["fp16", "fp32"]), rng.choice(["fp16", "fp32"])).items()
                if k != "name"}
    seqs = rng.choice([1, 2, 3, 8, 16, 31])
    longest = _log(rng, 16, min(65536, 16 * 32768 * 8 * 128 // 2 // (seqs * heads * dim)))
    shortest = max(1, int(longest * rng.choice([0.05, 0.5, 1.0])))
    new = rng.choice([1, 1, 1, 2, 3, 5])
    per = rng.choice([1, 2, 4, 7, 8])
    return {k: v for k, v in _attend("", seqs, max(shortest, new), max(longest, new), new, heads * per, heads, dim,
                                     group, page).items() if k != "name"}


def _lens(case):
    """Cached tokens of each sequence after the step, from the case alone."""
    n = case["seqs"]
    if case["op"] == "cache":
        return [case["past"] + case["new"]] * n
    lo, hi = case["shortest"], case["longest"]
    return [hi - (hi - lo) * ((i * 7) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
_SIZE = {"fp16": 2, "fp32": 4}


def work(case):
    if case["op"] == "product":
        M, K, B = case["M"], case["K"], case["batch"]
        meta = {"uniform": M * (K // 16) * 4, "lut": M * (2 << case["bits"])}.get(case["fmt"])
        if meta is None:
            meta = M * (K // case["group"]) * (case["bits"] + 1) * 2
        nnz = int(M * K * case["density"])
        mo = M // 2 if case["gated"] else M
        b = M * K * case["bits"] // 8 + meta + 6 * nnz + 4 * (M + 1) + 2 * B * K + _SIZE[case["out"]] * B * mo
        b += (2 * M if case["bias"] else 0) + (2 * B * mo if case["residual"] else 0)
        return {"bytes": b, "flops": 2 * B * (M * K + nnz)}
    per = case["heads"] * (case["dim"] // 2 + 4 * (case["dim"] // case["group"])) * 2  # keys and values of a token
    if case["op"] == "cache":
        t = case["seqs"] * case["new"]
        el = 2 * t * case["heads"] * case["dim"]
        # values in, codes and statistics out, the same codes in, values out
        return {"bytes": el * (_SIZE[case["dtype"]] + _SIZE[case["out"]]) + 2 * t * per, "flops": 8 * el}
    t, lens = case["seqs"] * case["new"], _lens(case)
    rows = case["new"] * case["q_heads"]
    return {"bytes": sum(lens) * per + 4 * t * case["q_heads"] * case["dim"],
            "flops": 4 * rows * case["dim"] * sum(lens)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * seed + sum(ord(c) * (i + 1) for i, c in enumerate(repr(sorted(
        (k, v) for k, v in case.items() if k != "name")))) % 1000003)
    return g


def _product_inputs(case, seed):
    """The canonical arrays of one weight set, x, bias and residual, on the GPU."""
    g = _gen(case, seed)
    M, K, B, bits = case["M"], case["K"], case["batch"], case["bits"]

    def uni(shape, lo, hi):
        return torch.rand(shape, generator=g, device=DEV) * (hi - lo) + lo

    w = {"codes_packed": torch.randint(0, 256, (M, K * bits // 8), generator=g, device=DEV, dtype=torch.uint8)}
    top = (1 << bits) - 1
    if case["fmt"] == "uniform":
        w["scales"] = (uni((M, K // 16), 0.5, 1.5) * 0.08 / top).half()
        w["zeros"] = torch.randint(0, top + 1, (M, K // 16), generator=g, device=DEV).half()
    elif case["fmt"] == "lut":
        lut = torch.randn((M, top + 1), generator=g, device=DEV) * 0.03
        lut[:, 0] = 0
        w["lut"] = lut.half().sort(dim=1).values
    else:
        G = K // case["group"]
        step = torch.tensor([1.0, 2.0, 4.0], device=DEV) * 0.02
        w["coefs"] = torch.cat([-uni((M, G, 1), 3.0, 4.0) * 0.02, uni((M, G, 3), 0.5, 1.5) * step], dim=2).half()
    nnz = int(M * K * case["density"])
    pos = torch.randint(0, M * K, (nnz,), generator=g, device=DEV).unique()  # ascending, a few fewer than drawn
    w["rows"], w["cols"] = pos // K, pos % K
    sign = torch.randint(0, 2, pos.shape, generator=g, device=DEV) * 2 - 1
    w["values"] = (uni(pos.shape, 0.2, 2.5) * sign).half()
    x = torch.randn((B, K), generator=g, device=DEV).half()
    bias = torch.randn(M, generator=g, device=DEV).half() if case["bias"] else None
    mo = M // 2 if case["gated"] else M
    residual = torch.randn((B, mo), generator=g, device=DEV).half() if case["residual"] else None
    return w, x, bias, residual


def _canonical(case, w):
    """The same arrays as the package's descriptor takes them: host arrays, CSR rows."""
    M = case["M"]
    out = {"M": M, "K": case["K"], "bits": case["bits"], "fmt": case["fmt"], "group": case["group"]}
    for k in ("codes_packed", "scales", "zeros", "lut", "coefs"):
        if k in w:
            out[k] = w[k].cpu().numpy()
    counts = torch.bincount(w["rows"], minlength=M).cpu().numpy()
    out["row_ptr"] = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out["col_idx"] = w["cols"].cpu().numpy().astype(np.int32)
    out["values"] = w["values"].cpu().numpy()
    return out


def _pages(case, lens, g):
    """Page table [sequences, pages] over a pool with a few spare pages, in shuffled order; -1 behind the last."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, total


def _cache_inputs(case, seed):
    g = _gen(case, seed)
    H, D, t = case["heads"], case["dim"], case["seqs"] * case["new"]
    lens = _lens(case)
    table, total = _pages(case, lens, g)
    dt = {"fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]
    # keys sit around an offset per channel, values around zero
    k = torch.randn((t, H, D), generator=g, device=DEV) + 2 * torch.randn((H, D), generator=g, device=DEV)
    v = torch.randn((t, H, D), generator=g, device=DEV)
    return k.to(dt), v.to(dt), lens, table, total


def _attend_inputs(case, seed):
    """Queries, and the keys and values [tokens, heads, dim] of all sequences, one after another."""
    g = _gen(case, seed)
    H, D = case["heads"], case["dim"]
    lens = _lens(case)
    table, total = _pages(case, lens, g)
    off = 2 * torch.randn((H, D), generator=g, device=DEV)
    ks, vs = [], []
    for n in lens:
        ks.append((torch.randn((n, H, D), generator=g, device=DEV) + off).half())
        vs.append(torch.randn((n, H, D), generator=g, device=DEV).half())
    q = (2 * torch.randn((case["seqs"] * case["new"], case["q_heads"], D), generator=g, device=DEV)).half()
    return q, torch.cat(ks), torch.cat(vs), lens, table, total


def _slots(lens, new, table, page):
    """Pool slot of each of the last `new[s]` positions of every sequence."""
    out = []
    for s, n in enumerate(lens):
        p = torch.arange(n - new[s], n, device=DEV)
        out.append(table[s].long()[p // page] * page + p % page)
    return torch.cat(out)


def _starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def prepare(case, seed):
    if case["op"] == "product":
        w, x, bias, residual = _product_inputs(case, seed)
        st = {"case": case, "x": x, "bias": bias, "residual": residual}
        if own:
            from dense_sparse_bit_amd import qgemv
            st["plan"] = qgemv.QGemv(_canonical(case, w))
        else:
            st["w"] = w
        return st
    H, D, G, page = case["heads"], case["dim"], case["group"], case["page"]
    if case["op"] == "cache":
        k, v, lens, table, total = _cache_inputs(case, seed)
        new = [case["new"]] * case["seqs"]
        st = {"case": case, "k": k, "v": v, "pages": table}
        if own:
            from dense_sparse_bit_amd import qcache
            st["cache"] = qcache.QCache(total, H, D, page_size=page, group=G)
            st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
            st["q_start"] = None if case["new"] == 1 else _starts(new)
        else:
            st["slots"] = _slots(lens, new, table, page)
            st["pool"] = _pool(total * page, H, D, G)
        return st
    q, k, v, lens, table, total = _attend_inputs(case, seed)
    st = {"case": case, "q": q, "pages": table, "scale": 1 / math.sqrt(D)}
    if own:
        from dense_sparse_bit_amd import qcache
        st["cache"] = qcache.QCache(total, H, D, page_size=page, group=G)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["cache"].write(k, v, st["lens"], table, _starts(lens))
        st["q_start"] = None if case["new"] == 1 else _starts([case["new"]] * case["seqs"])
    else:
        st["lens"] = lens
        st["pool"] = _pool(total * page, H, D, G)
        at = 0
        for s, n in enumerate(lens):
            sl = _slots([n], [n], table[s:s + 1], page)
            _plain_write(st["pool"], sl, k[at:at + n], v[at:at + n], G)
            at += n
        st["slots"] = [_slots([n], [n], table[s:s + 1], page) for s, n in enumerate(lens)]
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_weights(case, w):
    """Dense fp32 W [M, K]: codes from the bitstreams, decoded, plus the outliers."""
    M, K, bits = case["M"], case["K"], case["bits"]
    p = w["codes_packed"]
    if bits == 4:
        q = torch.stack([p & 15, p >> 4], dim=2).view(M, K)
    else:
        t = p.view(M, K // 8, 3).int()
        t = t[:, :, 0] | (t[:, :, 1] << 8) | (t[:, :, 2] << 16)
        q = torch.stack([((t >> (3 * j)) & 7).to(torch.uint8) for j in range(8)], dim=2).view(M, K)
    if case["fmt"] == "uniform":
        W = (q.view(M, K // 16, 16).float() - w["zeros"].float()[:, :, None]) * w["scales"].float()[:, :, None]
    elif case["fmt"] == "lut":
        W = torch.gather(w["lut"].float(), 1, q.long())
    else:
        c = w["coefs"].float()
        qg = q.view(M, K // case["group"], case["group"])
        W = c[:, :, 0:1].expand(qg.shape).clone()
        for t in range(bits):
            W += c[:, :, t + 1:t + 2] * ((qg >> t) & 1).float()
    W = W.reshape(M, K)
    W[w["rows"], w["cols"]] += w["values"].float()
    return W


def _plain_act(t, act):
    if act == "relu":
        return torch.where(t > 0, t, torch.zeros_like(t))
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return 0.5 * t * (1 + torch.erf(t * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * t * (1 + torch.tanh(0.7978845608028654 * (t + 0.044715 * t * t * t)))
    return t


def _plain_product(st):
    case = st["case"]
    t = st["x"].float() @ _plain_weights(case, st["w"]).t()
    if st["bias"] is not None:
        t = t + st["bias"].float()
    if case["gated"]:
        t = _plain_act(t[:, 0::2], case["act"]) * t[:, 1::2]
    else:
        t = _plain_act(t, case["act"])
    if st["residual"] is not None:
        t = t + st["residual"].float()
    return t.half() if case["out"] == "fp16" else t


def _pool(slots, H, D, G):
    """Plain 4-bit storage of keys and values: codes, step and lowest value per group."""
    return [{"q": torch.zeros((slots, H, D // 2), dtype=torch.uint8, device=DEV),
             "s": torch.zeros((slots, H, D // G), dtype=torch.float16, device=DEV),
             "lo": torch.zeros((slots, H, D // G), dtype=torch.float16, device=DEV)} for _ in range(2)]


def _plain_write(pool, slots, k, v, G):
    for st, val in zip(pool, (k, v)):
        t, H, D = val.shape
        x = val.half().float().view(t, H, D // G, G)
        lo = x.amin(dim=3)
        s = ((x.amax(dim=3) - lo) / 15).half()
        q = torch.round((x - lo[..., None]) / s.float()[..., None])
        q = torch.where(s[..., None] > 0, q, torch.zeros_like(q)).clamp(0, 15).to(torch.uint8).view(t, H, D)
        st["q"][slots] = q[..., 0::2] | (q[..., 1::2] << 4)
        st["s"][slots] = s
        st["lo"][slots] = lo.half()


def _plain_read(st, slots, G):
    p = st["q"][slots]
    t, H, D = p.shape[0], p.shape[1], 2 * p.shape[2]
    q = torch.stack([p & 15, p >> 4], dim=3).view(t, H, D // G, G).float()
    return (q * st["s"][slots].float()[..., None] + st["lo"][slots].float()[..., None]).view(t, H, D)


def _plain_cache(st):
    case = st["case"]
    _plain_write(st["pool"], st["slots"], st["k"], st["v"], case["group"])
    dt = {"fp16": torch.float16, "fp32": torch.float32}[case["out"]]
    return tuple(_plain_read(p, st["slots"], case["group"]).to(dt) for p in st["pool"])


def _plain_attend(st):
    case, q = st["case"], st["q"]
    H, D, n_new = case["heads"], case["dim"], case["new"]
    per = case["q_heads"] // H
    out = torch.empty_like(q)
    for s, n in enumerate(st["lens"]):
        k = _plain_read(st["pool"][0], st["slots"][s], case["group"]).permute(1, 2, 0).contiguous()  # [H, D, n]
        v = _plain_read(st["pool"][1], st["slots"][s], case["group"]).permute(1, 0, 2).contiguous()  # [H, n, D]
        qs = q[s * n_new:(s + 1) * n_new].float().view(n_new, H, per, D).permute(1, 0, 2, 3).reshape(H, n_new * per, D)
        sc = torch.matmul(qs, k) * st["scale"]
        pos = torch.arange(n, device=DEV)[None, :]
        last = n - n_new + torch.arange(n_new, device=DEV).repeat_interleave(per)[:, None]
        sc = torch.where(pos <= last, sc, torch.full_like(sc, -math.inf))
        p = torch.exp(sc - sc.amax(dim=2, keepdim=True))
        o = torch.matmul(p, v) / p.sum(dim=2, keepdim=True)
        out[s * n_new:(s + 1) * n_new] = o.view(H, n_new, per, D).permute(1, 0, 2, 3).reshape(n_new, H * per, D).half()
    return out


def run(state):
    case = state["case"]
    if not own:
        return {"product": _plain_product, "cache": _plain_cache, "attend": _plain_attend}[case["op"]](state)
    if case["op"] == "product":
        return state["plan"].run_epilogue(
            state["x"], bias=state["bias"], act=case["act"], gated=case["gated"], residual=state["residual"],
            dtype=torch.float16 if case["out"] == "fp16" else torch.float32)
    if case["op"] == "cache":
        state["cache"].write(state["k"], state["v"], state["lens"], state["pages"], state["q_start"])
        return state["cache"].read(state["lens"], state["pages"], state["q_start"], n_tok=state["k"].shape[0],
                                   dtype=torch.float16 if case["out"] == "fp16" else torch.float32)
    return state["cache"].attend(state["q"], state["lens"], state["pages"], state["q_start"], scale=state["scale"])


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def _exact_act(t, act):
    if act == "relu":
        return np.maximum(t, 0)
    if act == "silu":
        return t * np.exp(-np.logaddexp(0, -t))
    if act == "gelu":
        return t * np.vectorize(lambda z: 0.5 * math.erfc(-z / math.sqrt(2)))(t)
    if act == "gelu_tanh":
        return t * 0.5 * (1 + np.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
    return t


def _exact_product(case, seed):
    w, x, bias, residual = _product_inputs(case, seed)
    M, K, bits = case["M"], case["K"], case["bits"]
    packed = w["codes_packed"].cpu().numpy()
    x64 = x.cpu().numpy().astype(np.float64)
    meta = {k: w[k].cpu().numpy().astype(np.float64) for k in ("scales", "zeros", "lut", "coefs") if k in w}
    y = np.empty((x64.shape[0], M))
    step = max(1, (1 << 24) // K)
    weigh = 1 << np.arange(bits, dtype=np.uint8)
    for r in range(0, M, step):
        e = min(M, r + step)
        planes = np.unpackbits(packed[r:e], axis=1, bitorder="little").reshape(e - r, K, bits)
        if case["fmt"] == "bpdq":
            c = np.repeat(meta["coefs"][r:e], case["group"], axis=1)
            d = c[:, :, 0] + (c[:, :, 1:] * planes).sum(axis=2)
        else:
            q = (planes * weigh).sum(axis=2, dtype=np.int64)
            if case["fmt"] == "lut":
                d = np.take_along_axis(meta["lut"][r:e], q, axis=1)
            else:
                d = np.repeat(meta["scales"][r:e], 16, axis=1) * (q - np.repeat(meta["zeros"][r:e], 16, axis=1))
        y[:, r:e] = x64 @ d.T
    rows, cols = w["rows"].cpu().numpy(), w["cols"].cpu().numpy()
    vals = w["values"].cpu().numpy().astype(np.float64)
    for b in range(x64.shape[0]):
        y[b] += np.bincount(rows, weights=vals * x64[b, cols], minlength=M)
    if bias is not None:
        y += bias.cpu().numpy().astype(np.float64)
    if case["gated"]:
        y = _exact_act(y[:, ::2], case["act"]) * y[:, 1::2]
    else:
        y = _exact_act(y, case["act"])
    if residual is not None:
        y += residual.cpu().numpy().astype(np.float64)
    return y


def _exact_values(v, G):
    """lo + s q of each value in 64 bits.  The storage is defined with FP16
    values, an FP16 step and a quotient of FP32, so those are kept."""
    t, H, D = v.shape
    x = v.half().double().view(t, H, D // G, G)
    lo, hi = x.min(dim=3, keepdim=True).values, x.max(dim=3, keepdim=True).values
    s = ((hi - lo).float() / 15).half()
    q = ((x - lo).float() / s.float()).double().round().clamp(0, 15)
    return (lo + torch.where(s > 0, s.double() * q, torch.zeros_like(q))).view(t, H, D)


def exact(case, seed):
    if case["op"] == "product":
        return _exact_product(case, seed)
    G = case["group"]
    if case["op"] == "cache":
        k, v, _, _, _ = _cache_inputs(case, seed)
        return _exact_values(k, G), _exact_values(v, G)
    q, k, v, lens, _, _ = _attend_inputs(case, seed)
    H, D, new = case["heads"], case["dim"], case["new"]
    per = case["q_heads"] // H
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    at = 0
    for s, n in enumerate(lens):
        for h in range(H):
            kh = _exact_values(k[at:at + n, h:h + 1], G)[:, 0]
            vh = _exact_values(v[at:at + n, h:h + 1], G)[:, 0]
            for i in range(new):
                m = n - new + i + 1
                a = q[s * new + i, h * per:(h + 1) * per].double() @ kh[:m].t().contiguous() / math.sqrt(D)
                out[s * new + i, h * per:(h + 1) * per] = torch.softmax(a, dim=1) @ vh[:m]
        at += n
    return out
