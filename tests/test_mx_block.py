"""A decoder block out of the operators between its norms: norm into MX blocks, stacked q/k/v product, rotary append to the
4-bit cache, attention, output product, norm with the residual stream, gated product, down product; prompts first, then single
tokens, captured.  Each operator is checked against fp64 from its own inputs, with its own tolerance (tests/test_qnorm.py,
test_qmx.py, test_qrotary.py, test_qcache.py)."""

import math

import numpy as np
import pytest

from dense_sparse_bit_amd import qcache, qmx, qnorm, qrotary
from gpu_checks import say
from oracle import block, mx
from oracle import cache as oc
from test_qcache import Batch, check_attend
from test_qmx import check as check_product
from test_qnorm import check as check_norm
from test_qrotary import check_turned, freqs

pytestmark = pytest.mark.gpu

HQ, H, D, G, PAGE, E, F = 4, 2, 64, 32, 16, 256, 352


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class Block:
    def __init__(self, torch, fmt, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        shapes = {"qkv": ((HQ + 2 * H) * D, E), "o": (E, HQ * D), "gate_up": (2 * F, E), "down": (E, F)}
        self.w = {n: qmx.QMx(qmx.quantize(torch.randn(s, generator=g, device="cuda") / math.sqrt(s[1]))) for n, s in shapes.items()}
        self.values = {n: host(p.w.values()) for n, p in self.w.items()}
        self.n1, self.n2 = ((1 + 0.2 * torch.randn(E, generator=g, device="cuda")).half() for _ in range(2))
        self.rotary = qrotary.Rotary(freqs(D))
        self.fmt = fmt

    def run(self, h, cache, lens, pages, start=None):
        """Every operator's output, by name."""
        r = {}
        _, r["x1"] = qnorm.norm(None, h, pre=self.n1, out_type=self.fmt, keep_h=False)
        r["qkv"] = self.w["qkv"].run(r["x1"])
        q, k, v = (t.unflatten(1, (-1, D)) for t in r["qkv"].split([HQ * D, H * D, H * D], dim=1))
        r["q"], r["k"], r["v"] = q, k, v
        r["turned"] = self.rotary.write(cache, q, k, v, lens, pages, start)
        r["a"] = cache.attend(r["turned"], lens, pages, start)
        r["o"] = self.w["o"].run(r["a"].flatten(1), self.fmt)
        r["h2"], r["x2"] = qnorm.norm(r["o"], h, pre=self.n2, out_type=self.fmt)
        r["m"] = self.w["gate_up"].run(r["x2"], act="silu", gated=True)
        r["y"] = self.w["down"].run(r["m"], self.fmt, residual=r["h2"])
        return r

    def check(self, torch, h, r, b, enc):
        """enc: what the cache holds of each sequence's keys and values, extended by the call's own."""
        _, (o, do) = block.norm(None, host(h), pre=host(self.n1))
        _, out = qnorm.norm(None, h, pre=self.n1, out_type="fp32")
        check_norm(out, o, do, "first norm")
        same = qmx.quantize(out, self.fmt)
        assert all(torch.equal(x, y) for x, y in zip(same.unpack(), r["x1"].unpack()))
        check_product(r["qkv"], *mx.product(host(r["x1"].values()), self.values["qkv"]), False)
        own = np.concatenate([b.positions(s) for s in range(len(b.lens))])[None]
        check_turned(r["turned"], r["q"].cpu().numpy(), own, self.rotary.freqs.cpu().numpy(), "halves")
        k = self.rotary.write(qcache.QCache(b.total, H, D, page_size=PAGE, group=G), r["k"].contiguous(), r["k"], r["v"], *b.args())
        for s in range(len(b.lens)):
            rows = slice(b.start[s], b.start[s + 1])
            for i, new in enumerate((k, r["v"])):
                e = oc.quantise(new[rows].cpu().numpy(), G)
                for key in e:
                    enc[s][i][key] = np.concatenate([enc[s][i][key], e[key]]) if enc[s][i] and key in enc[s][i] else e[key]
        check_attend(b, enc, r["turned"].cpu().numpy(), r["a"], 1 / math.sqrt(D), "attention")
        a = mx.values(*mx.quantise(r["a"].flatten(1).cpu().numpy(), self.fmt), self.fmt)
        check_product(r["o"], *mx.product(a, self.values["o"]), False)
        (h2, dh), (x2, dx) = block.norm(host(r["o"]), host(h), pre=host(self.n2))
        check_norm(r["h2"], h2, dh, "stream")
        _, out = qnorm.norm(r["o"], h, pre=self.n2, out_type="fp32")
        check_norm(out, x2, dx, "second norm")
        same = qmx.quantize(out, self.fmt)
        assert all(torch.equal(x, y) for x, y in zip(same.unpack(), r["x2"].unpack()))
        check_product(r["m"], *mx.product(host(r["x2"].values()), self.values["gate_up"], act="silu", gated=True), False)
        m = mx.values(*mx.quantise(r["m"].cpu().numpy(), self.fmt), self.fmt)
        check_product(r["y"], *mx.product(m, self.values["down"], residual=host(r["h2"])), False)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("prompts", [[5], [40, 1, 17], [33] * 9, [300, 70]])
def test_prompts_and_steps(torch, prompts, fmt):
    blk = Block(torch, fmt)
    S = len(prompts)
    last = [n + 2 for n in prompts]
    full = Batch(torch, last, [1] * S, PAGE, seed=S, one_each=True)  # pages for the steps too
    cache = qcache.QCache(full.total, H, D, page_size=PAGE, group=G)
    enc = [({}, {}) for _ in prompts]
    say(f"[gpu] block, prompts {prompts}, {fmt}")
    for lens, new in [(prompts, prompts), ([n + 1 for n in prompts], [1] * S), (last, [1] * S)]:
        b = Batch(torch, lens, new, PAGE, seed=S, one_each=new[0] == 1 and lens != prompts)
        b.d_pages, b.total, b.table = full.d_pages, full.total, full.table
        h = torch.randn((sum(new), E), device="cuda").half()
        r = blk.run(h, cache, *b.args())
        blk.check(torch, h, r, b, enc)


def test_captured_steps(torch):
    """A step of three sequences captured once and replayed for the tokens that follow, against eager steps."""
    blk = Block(torch, "e4m3", seed=3)
    S = 3
    h = torch.randn((S, E), device="cuda").half()
    pages = torch.arange(12, dtype=torch.int32, device="cuda").view(S, 4)
    lens = torch.tensor([9, 30, 17], dtype=torch.int32, device="cuda")
    one, two = (qcache.QCache(12, H, D, page_size=PAGE, group=G) for _ in range(2))
    k = torch.randn((int(lens.sum()), H, D), device="cuda").half()
    start = torch.tensor([0, 9, 39, 56], dtype=torch.int32, device="cuda")
    for c in (one, two):
        c.data.zero_()
        c.write(k, k, lens, pages, start)
    blk.run(h, qcache.QCache(12, H, D, page_size=PAGE, group=G), lens, pages)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = blk.run(h, one, lens, pages)
    for _ in range(5):
        lens += 1
        h.normal_()
        g.replay()
        want = blk.run(h, two, lens, pages)
        torch.cuda.synchronize()
        assert torch.equal(one.data, two.data)
        for n in ("qkv", "turned", "a", "o", "h2", "m", "y"):
            assert torch.equal(r[n], want[n]), n
