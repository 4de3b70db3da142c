"""Attention whose ranges are long, and whose sequences are many, where ranges are cut inside items.

A workgroup takes one range of all items' blocks of 128 positions.  Here
ranges hold more than 32 blocks of one item (a wave then looks its pages up
again, and its two tiles of LDS go round many times), and calls have up to 200
ragged sequences (several rounds of 64 lengths) whose items several workgroups
share.

All sequences use the same pages, each in an order of its own, some of them
missing.  Values are one page's own number in one of its own dimensions, so a
page left out, read twice or from elsewhere changes an output by far more than
the tolerance.  All values are positive, so the tolerance is relative to the
output: values and output FP16 (2^-11 each), weights 2^-22, exp2 2^-22, scores
(2^-18 + 2^-23) of B = scale sum |q| (|lo| + 15 s), numerator and denominator
each; fp32 sums (L / 32 + 16) 2^-24 each; weights below FP16's range 2^-32 of
the largest.
"""

import ctypes
import math

import numpy as np
import pytest

from dense_sparse_bit_amd import qcache
from gpu_checks import say
from oracle import cache as oc
from test_qcache import Batch, fill

ITEM_COST = 3  # blocks that an item's start and end count as


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


class Call:
    def __init__(self, D, G, page, H, per, lens, new, seed):
        self.D, self.G, self.page, self.H, self.per, self.lens, self.new, self.seed = D, G, page, H, per, lens, new, seed
        self.S, self.n_tok = len(lens), sum(new) + 2  # two rows of padding
        self.max_pages = -(-max(lens) // page)
        rng = np.random.default_rng(seed)
        self.order = np.stack([rng.permutation(self.max_pages) for _ in range(self.S)])
        self.hole = rng.random((self.S, self.max_pages)) < 0.04
        self.q = (0.7 * rng.standard_normal((self.n_tok, H * per, D))).astype(np.float16)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)

    def grid(self):
        """Workgroups, from the workspace: two partials of 16 rows and 16 bytes for each."""
        sh = qcache.Shape(self.max_pages, self.H, self.D, self.page, self.G)
        sq, n = qcache.Seqs(self.S, self.n_tok, self.max_pages, 4096, 4096, 4096), ctypes.c_size_t(0)
        assert qcache.lib().qcache_attend_ws(sh, sq, self.H * self.per, n) == 0
        each = 2 * 16 * (self.D + 4) * 4 + 16
        assert n.value % each == 0
        return n.value // each

    def items(self):
        """Blocks of every item, in order."""
        return [nb for L, n in zip(self.lens, self.new) for nb in [-(-max(L, 0) // 128)] if nb
                for _ in range(-(-n * self.per // 16) * self.H)]

    def longest_runs(self):
        """Of every range, the most consecutive blocks of one item."""
        nbs = np.array(self.items())
        ends = np.cumsum(nbs + ITEM_COST)
        total, grid = int(ends[-1]), self.grid()
        q, rem = divmod(total, min(grid, total))
        runs = []
        for g in range(min(grid, total)):
            a, b = g * q + min(g, rem), (g + 1) * q + min(g + 1, rem)
            i, best = int(np.searchsorted(ends, a, side="right")), 0
            while i < len(nbs) and ends[i] - nbs[i] - ITEM_COST < b:
                first = ends[i] - nbs[i] - ITEM_COST
                best = max(best, min(b, first + nbs[i]) - max(a, first))
                i += 1
            runs.append(best)
        return np.array(runs)


def long_call(D, G, page, H, per, S):
    rng = np.random.default_rng(D)
    return Call(D, G, page, H, per, rng.integers(9500, 10302, S).tolist(), [1] * (S - 1) + [2], D)


def ragged_call(S, D, G, page, H, per):
    rng = np.random.default_rng(S)
    lens = [int(x) if rng.random() < 0.9 else int(rng.integers(-3, 1)) for x in rng.integers(1, 2600, S)]
    new = rng.choice([0, 1, 1, 1, 2, 3], S).tolist()
    lens[S // 2], new[S // 2] = 2601, 3  # the table's width, and rows enough for two tiles of 8 heads
    return Call(D, G, page, H, per, lens, new, S)


LONG = [(256, 64, 16, 2, 2, 126), (128, 32, 64, 2, 3, 188), (64, 64, 32, 4, 1, 126)]
RAGGED = [(70, 128, 32, 64, 2, 8), (130, 64, 32, 16, 1, 5), (200, 256, 128, 32, 2, 3), (129, 128, 64, 16, 3, 8)]


@pytest.mark.parametrize("args", LONG)
def test_long_calls_pass_32_blocks(args):
    """What the long calls are for: most ranges hold 34 or more blocks of one item."""
    runs = long_call(*args).longest_runs()
    assert (runs >= 34).mean() > 0.5


@pytest.mark.parametrize("args", RAGGED)
def test_ragged_calls_are_cut(args):
    """Items lie in several ranges: more blocks than four a sequence, and ranges shorter than the longest items."""
    call = ragged_call(*args)
    runs, nbs = call.longest_runs(), call.items()
    assert call.S > 64 and call.max_pages * call.page > 4 * 128
    assert max(nbs) > 2 * np.median(runs)


def attend_and_check(torch, call, what):
    H, D, page, per = call.H, call.D, call.page, call.per
    n = call.max_pages
    base = Batch(torch, [n * page], [1], page, seed=call.seed)
    p = np.arange(n * page) // page

    def vals(_, v):
        v = np.zeros_like(v)
        for h in range(H):
            v[np.arange(n * page), h, (p + 5 * h) % D] = 1 + p // D
        return v

    c, ((ek, ev),) = fill(torch, base, H, D, call.G, seed=call.seed, vals=vals)
    table = np.where(call.hole, -1, base.table[0][call.order]).astype(np.int32)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    q = cu(call.q)
    mark = torch.full(q.shape, -7.5, dtype=torch.float16, device="cuda")
    args = (cu(np.array(call.lens, np.int32)), cu(table), cu(call.start))
    say(f"[gpu] attend {what} D={D} G={call.G} page={page} heads={H} x {per}, {call.S} sequences")
    got = c.attend(q, *args, out=mark.clone())
    assert torch.equal(got[call.start[-1]:], mark[call.start[-1]:]), "padding rows were written"
    assert torch.equal(c.attend(q, *args)[:call.start[-1]], got[:call.start[-1]]), "not bitwise deterministic"

    K, W = (cu(oc.values(e)).view(n, page, H, D) for e in (ek, ev))
    reach, scale = cu(oc.reach(ek)).amax(dim=0), 1 / math.sqrt(D)
    got, q = got.double(), q.double()
    top = float(W.max())
    worst = 0.0
    for s, (L, m) in enumerate(zip(call.lens, call.new)):
        r0 = int(call.start[s])
        if m == 0:
            continue
        if L <= 0:
            assert not got[r0:r0 + m].any()
            continue
        order = torch.from_numpy(call.order[s]).cuda()
        pos = torch.arange(n * page, device="cuda")
        there = torch.from_numpy(~call.hole[s]).cuda()[pos // page]
        see = there[None] & (pos[None] <= torch.arange(L - m, L, device="cuda")[:, None])  # [rows, positions]
        for h in range(H):
            k, v = K[order, :, h].reshape(-1, D), W[order, :, h].reshape(-1, D)
            for i in range(m):
                x = q[r0 + i, h * per:(h + 1) * per]
                y = got[r0 + i, h * per:(h + 1) * per]
                if not bool(see[i].any()):
                    assert not y.any()
                    continue
                a = (x @ k[see[i]].t().contiguous()) * scale
                want = torch.softmax(a, dim=1) @ v[see[i]]
                B = scale * (x.abs() @ reach[h])[:, None]
                rel = 2 * 2.0 ** -11 + 2 * ((2.0 ** -18 + 2.0 ** -23) * B + 2 * 2.0 ** -22) + 2 * (L / 32 + 16) * 2.0 ** -24
                tol = rel * want + L * 2.0 ** -32 * top + 2.0 ** -25
                worst = max(worst, float(((y - want).abs() / tol).max()))
                assert worst <= 1, f"sequence {s}, row {i}, head {h}: {worst:.2f} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("args", LONG)
def test_ranges_past_32_blocks(torch, args):
    attend_and_check(torch, long_call(*args), "long ranges")


@pytest.mark.gpu
@pytest.mark.parametrize("args", RAGGED)
def test_many_sequences_cut_inside_items(torch, args):
    attend_and_check(torch, ragged_call(*args), "many ragged sequences")
