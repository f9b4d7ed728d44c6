"""Attention of a batch that shares prefixes, on the GPU against the oracle.

Tolerances.  O: a weight of P is rounded to bf16 (half a step, 2^-8 of it) and
so is the result, which gives |error| <= 2^-8 (sum_j p_j |v_j| + |o|) element
by element, plus 2^-13 (of values up to about 4) for the fp32 sums and
exponentials.  LSE: a score's fp32 sum of 128 products of normal variables is
off by at most 128 * 2^-24 * sum |q_i k_i| * scale < 1e-4; 2e-4 with the
exponentials' 2^-22 and the final logarithm."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from sparse_kv_verification_gb300 import build, inputs as I, native as N
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE_RANGE = 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return N.load()


def flags():
    f = ctypes.c_uint32(0)
    N.load().dustin_device_status(ctypes.byref(f))
    return f.value


class Case:
    """Inputs on the CPU, caches on the GPU (paged: one pool, shuffled, its
    unused rows NaN)."""

    def __init__(self, b, groups, hq, hkv, d, w, n_p, n_o, page=0, win=True, prefix_len=None,
                 own_len=None, seed=0, garbage=float("nan")):
        g = I.generator(seed)
        r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
        self.__dict__.update(b=b, groups=groups, hkv=hkv, n_p=n_p, n_o=n_o, d=d, page=page,
                             scale=d ** -0.5, prefix_len=prefix_len, own_len=own_len)
        self.q = r(b, hq, w, d)
        self.kv = [[r(groups, hkv, n_p, d), r(groups, hkv, n_p, d)],
                   [r(b, hkv, n_o, d), r(b, hkv, n_o, d)]]
        self.win = [r(b, hkv, w, d), r(b, hkv, w, d)] if win else None
        lens = [prefix_len or [n_p] * groups, own_len or [n_o] * b]
        stored = [[x.clone() for x in kv] for kv in self.kv]
        for kv, ln in zip(stored, lens):
            for x in kv:
                for i, n in enumerate(ln):
                    x[i, :, max(n, 0):] = garbage
        self.tables = [None, None]
        if page:
            pp, po = -(-n_p // page), -(-n_o // page)
            perm = torch.randperm(groups * pp + b * po + 2, generator=g).int()
            # Sequences' rows as after a fork: their own pages follow the
            # places of the shared ones.
            rows = torch.full((b, pp + po), 1 << 30, dtype=torch.int32)
            rows[:, pp:] = perm[groups * pp:groups * pp + b * po].view(b, po)
            self.tables = [perm[:groups * pp].view(groups, pp).to(DEV), rows.to(DEV)[:, pp:]]
            pools = []
            for x in range(2):
                pool = torch.full((len(perm), hkv, page, d), garbage, dtype=torch.bfloat16)
                for kv, t in zip(stored, (perm[:groups * pp].view(groups, pp), rows[:, pp:])):
                    n, m = kv[x].shape[2], t.shape[1]
                    padded = torch.full((kv[x].shape[0], hkv, m * page, d), garbage,
                                        dtype=torch.bfloat16)
                    padded[:, :, :n] = kv[x]
                    pool[t.long()] = padded.view(len(t), hkv, m, page, d).transpose(1, 2)
                pools.append(pool.to(DEV))
            self.stored = [pools, pools]
        else:
            self.stored = [[x.to(DEV) for x in kv] for kv in stored]
        self.dev_win = None if self.win is None else [x.to(DEV) for x in self.win]

    def args(self):
        """Everything of a call but q, o, lse and the workspace."""
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)
        caches = [N.kv_desc(*kv, t) if n else None
                  for kv, t, n in zip(self.stored, self.tables, (self.n_p, self.n_o))]
        return dict(prefix=caches[0], own=caches[1], h_kv=self.hkv, groups=self.groups,
                    n_prefix=self.n_p, n_own=self.n_o, scale=self.scale,
                    prefix_len=i32(self.prefix_len), own_len=i32(self.own_len),
                    win=None if self.win is None else N.kv_desc(*self.dev_win))

    def workspace(self):
        b, hq, w, d = self.q.shape
        ws = N.workspace(N.dustin_prefix_verify_attn_workspace_size(
            b, self.groups, hq, self.hkv, d, w, self.n_p, self.n_o), DEV)
        return ws.fill_(255)

    def run(self, **kw):
        q = self.q.to(DEV)
        o = torch.full_like(q, float("nan"))
        lse = torch.full(q.shape[:3], float("nan"), device=DEV)
        N.dustin_prefix_verify_attn(q=q, o=o, lse=lse, ws=self.workspace(), **{**self.args(), **kw})
        H.sync()
        return o, lse

    def oracle(self, q=None, kv=None):
        f = lambda x: x.double().numpy()
        q = f(self.q) if q is None else q
        kv = kv or [[f(x) for x in c] for c in self.kv]
        win = [None, None] if self.win is None else [f(x) for x in self.win]

        def at(v_of):
            return S.prefix_attention(q, kv[0][0], v_of(kv[0][1]), kv[1][0], v_of(kv[1][1]),
                                      self.groups, self.scale, self.prefix_len, self.own_len,
                                      win[0], None if win[1] is None else v_of(win[1]))
        o, lse = at(lambda v: v)
        return o, lse, at(np.abs)[0]

    def check(self, got=None, **kw):
        o, lse = got or self.run()
        want_o, want_lse, spread = self.oracle(**kw)
        err = np.abs(H.f64(o) - want_o)
        bound = 2.0 ** -8 * (spread + np.abs(want_o)) + 2.0 ** -13
        assert np.all(err <= bound), (float(err.max()), float((err - bound).max()))
        seen = np.isfinite(want_lse)
        np.testing.assert_array_equal(np.isfinite(H.f64(lse)), seen)
        np.testing.assert_allclose(H.f64(lse)[seen], want_lse[seen], atol=2e-4, rtol=0)
        assert np.all(np.isneginf(H.f64(lse)[~seen])) and not H.f64(o)[~seen].any()
        return o, lse


SHAPES = [  # b, groups, h_q, h_kv, d, w, n_prefix, n_own
    (1, 1, 1, 1, 64, 1, 1, 1),
    (2, 1, 4, 2, 64, 4, 256, 32),
    (3, 1, 8, 2, 128, 5, 700, 131),
    (4, 2, 14, 2, 64, 4, 129, 65),
    (6, 3, 10, 2, 128, 3, 1000, 200),
    (13, 1, 8, 1, 128, 2, 513, 40),        # a pair of row tiles
    (11, 1, 16, 2, 64, 5, 385, 127),       # three and a half row tiles
    (2, 1, 33, 1, 128, 5, 300, 260),       # more than 128 rows of one sequence
    (1, 1, 64, 1, 64, 8, 90, 900),         # four row tiles of one sequence
    (2, 2, 2, 1, 128, 130, 70, 50),        # a window beyond one tile
    (1, 1, 8, 8, 128, 1, 5000, 0),         # nothing of its own
    (5, 5, 4, 4, 64, 1, 0, 333),           # no prefix
]


@pytest.mark.parametrize("page", [0, 16, 48, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_parity(shape, page):
    Case(*shape, page=page, seed=sum(shape) + page).check()
    assert flags() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 64])
def test_lengths_and_what_lies_behind_them(d, page):
    """Lengths at and around tile borders, zero, and beyond the limit; NaN in
    every row behind them (and in no other)."""
    Case(12, 2, 4, 2, d, 3, 400, 257, page=page, prefix_len=[0, 385], seed=d + page,
         own_len=[0, 1, 127, 128, 129, 255, 256, 257, 16, 0, 47, 200]).check()
    Case(6, 3, 4, 1, d, 2, 300, 40, page=page, win=False, prefix_len=[1, 0, 299], seed=d,
         own_len=[0, 40, 0, 0, 17, 5]).check()      # sequences 2 and 3 see nothing
    c = Case(4, 2, 4, 1, d, 2, 130, 40, page=page, prefix_len=[500, -3], own_len=[-1, 41, 40, 7],
             seed=d)
    c.check()                                       # clamped
    assert flags() == 0


def test_nothing_at_all():
    o, lse = Case(3, 1, 4, 2, 64, 2, 0, 0, win=False).check()
    o, lse = Case(3, 3, 4, 2, 128, 2, 200, 200, win=False, prefix_len=[0] * 3,
                  own_len=[0] * 3).check()
    Case(3, 1, 4, 2, 64, 2, 0, 0).check()           # the window alone


@pytest.mark.parametrize("garbage", [float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min])
def test_other_garbage_behind_the_lengths(garbage):
    Case(3, 1, 8, 2, 128, 2, 300, 150, page=16, prefix_len=[250], own_len=[3, 149, 0],
         garbage=garbage, seed=3).check()


def test_large_scores_and_a_rising_maximum():
    """Scores that grow along the positions move the running maximum through
    every tile; scores of several hundred do not overflow."""
    c = Case(2, 1, 4, 1, 128, 3, 1500, 300, seed=8)
    for kv in c.kv:
        n = kv[0].shape[2]
        kv[0].mul_(torch.linspace(0.1, 40.0, n).view(1, 1, n, 1).to(torch.bfloat16))
    c.stored = [[x.to(DEV) for x in kv] for kv in c.kv]
    o, lse = c.run()
    want_o, want_lse, spread = c.oracle()
    assert want_lse.max() > 100
    # Scores up to 40 times larger: their fp32 sums are off by up to 40e-4,
    # and weights by that factor too.
    assert np.all(np.abs(H.f64(o) - want_o) <= (2.0 ** -8 + 8e-3) * (spread + np.abs(want_o)) + 1e-3)
    np.testing.assert_allclose(H.f64(lse), want_lse, atol=4e-3, rtol=1e-6)


@pytest.mark.parametrize("order", ["rising", "falling", "shuffled"])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 40])
def test_scores_past_the_exponents_range(order, size):
    """Scores up to 2^87, whose fp32 steps are far larger than 1: the one
    largest score takes the whole row, its V exactly, and nothing loops or
    overflows.  Neighbouring keys differ by a step of bf16 (2^-8 of them at
    least), so no other score is within the range of an exponential."""
    c = Case(2, 1, 4, 1, 128, 2, 200, 0, win=False, seed=21)
    at = {"rising": torch.arange(200), "falling": torch.arange(200).flip(0),
          "shuffled": torch.randperm(200, generator=I.generator(5))}[order]
    # 200 neighbours of bf16 from 1 on, in that order
    keys = (torch.arange(200, dtype=torch.int32) + (0x3F80)).to(torch.int16).view(torch.bfloat16)
    c.q.fill_(size)
    c.kv[0][0] = (keys[at] * size).view(1, 1, 200, 1).expand(1, 1, 200, 128).contiguous()
    c.stored = [[x.to(DEV) for x in kv] for kv in c.kv]
    o, lse = c.run()
    best = int(at.argmax())
    want = c.kv[0][1][0, 0, best].to(DEV).expand_as(o)
    assert torch.equal(o, want)
    score = 128.0 * size * float(keys[-1]) * size * c.scale
    # The sum of 128 equal products, the scale, the maximum in base 2 and back
    # to base e: a rounding of 2^-24 each, of the scale's constant too.
    np.testing.assert_allclose(H.f64(lse), score, rtol=8 * 2.0 ** -24)


def test_cache_layouts():
    """[b][n][h][d] caches, one kv head's storage for all heads, one
    sequence's storage for all."""
    c = Case(4, 2, 4, 2, 64, 3, 300, 100, seed=2)
    c.stored = [[x.to(DEV).transpose(1, 2).contiguous().transpose(1, 2) for x in kv] for kv in c.kv]
    assert c.stored[0][0].stride(1) == 64
    first = c.check()
    wide = [[torch.full((x.shape[0], x.shape[1], x.shape[2] + 3, 72), float("nan"), device=DEV,
                        dtype=torch.bfloat16) for x in kv] for kv in c.kv]
    for kv, w in zip(c.kv, wide):
        for x, y in zip(kv, w):
            y[:, :, 1:-2, :64] = x.to(DEV)
    c.stored = [[y[:, :, 1:-2, :64] for y in w] for w in wide]
    for x, y in zip(first, c.run()):
        assert torch.equal(x, y)
    for dim in (0, 1):
        kv = [[x.narrow(dim, 0, 1).expand_as(x) for x in y] for y in c.kv]
        c.stored = [[x.narrow(dim, 0, 1).to(DEV).expand(x.shape) for x in y] for y in kv]
        assert c.stored[0][0].stride(dim) == 0
        c.check(kv=[[x.double().numpy() for x in y] for y in kv])


def test_bad_pages_are_left_out():
    page = 16
    c = Case(3, 1, 8, 2, 128, 2, 400, 100, page=page, seed=6)
    c.tables[0][0, 3], c.tables[0][0, 24], c.tables[1][1, 2] = -1, 1 << 29, 1 << 20
    o, lse = c.run()
    assert flags() == PAGE_RANGE
    f = lambda x: x.double().numpy().copy()
    keep_p = np.delete(np.arange(400), np.r_[48:64, 384:400])
    for i in range(3):
        keep_o = np.delete(np.arange(100), np.r_[32:48]) if i == 1 else np.arange(100)
        want, wl = S.prefix_attention(
            f(c.q[i:i + 1]), f(c.kv[0][0])[:, :, keep_p], f(c.kv[0][1])[:, :, keep_p],
            f(c.kv[1][0][i:i + 1])[:, :, keep_o], f(c.kv[1][1][i:i + 1])[:, :, keep_o], 1, c.scale,
            None, None, f(c.win[0][i:i + 1]), f(c.win[1][i:i + 1]))
        np.testing.assert_allclose(H.f64(o[i:i + 1]), want, atol=2e-2)
        np.testing.assert_allclose(H.f64(lse[i:i + 1]), wl, atol=2e-4)


def test_many_short_sequences():
    """More sequences than threads of a CTA, most of them a tile or nothing."""
    b = 900
    lens = torch.randint(0, 40, (b,), generator=I.generator(4)).tolist()
    lens[::7] = [0] * len(lens[::7])
    Case(b, 3, 2, 1, 64, 1, 50, 40, page=16, prefix_len=[50, 0, 31], own_len=lens, win=False,
         seed=9).check()


def test_equal_bits_other_stream_graph_and_workspace_reuse():
    """Equal calls give equal bits whatever the workspace held; captured, the
    call reads the lengths and caches of the time of the replay; two graphs
    share one workspace."""
    c = Case(7, 1, 8, 2, 128, 3, 2000, 300, page=16, own_len=[5, 300, 0, 77, 128, 130, 299], seed=5)
    o, lse = c.check()
    assert all(torch.equal(x, y) for x, y in zip((o, lse), c.run(flags=N.DUSTIN_ATTN_KV_READY)))
    ws, q, a = c.workspace(), c.q.to(DEV), c.args()
    outs = [(torch.empty_like(o), torch.empty_like(lse)) for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        N.dustin_prefix_verify_attn(q=q, o=outs[0][0], lse=outs[0][1], ws=ws, **a)
    side.synchronize()
    graphs = []
    for x in outs[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            N.dustin_prefix_verify_attn(q=q, o=x[0], lse=x[1], ws=ws, **a)
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    H.sync()
    for x in outs:
        assert torch.equal(x[0], o) and torch.equal(x[1], lse)
    c.own_len = [9, 1, 40, 0, 300, 256, 2]
    a["own_len"].copy_(torch.tensor(c.own_len))
    # Rows behind the first lengths hold NaN: give them values first.
    for x in range(2):
        for i in range(7):
            t = c.tables[1][i].long()
            got = torch.zeros((2, t.numel() * 16, 128), dtype=torch.bfloat16)
            got[:, :300] = c.kv[1][x][i]
            c.stored[1][x][t] = got.view(2, -1, 16, 128).transpose(0, 1).to(DEV)
    graphs[0].replay()
    H.sync()
    c.check(got=outs[1])


def test_long_prefix_against_fp64_on_the_gpu():
    """A prefix long enough that every CTA holds a part of one row tile's
    keys, and sequences enough for several row tiles."""
    c = Case(9, 1, 16, 1, 128, 5, 20000, 700, win=True, own_len=[700, 0, 1, 650, 3, 128, 127, 5, 99],
             seed=11)
    o, lse = c.run()
    f = lambda x: x.to(DEV).double()
    for i in range(9):
        k = torch.cat([f(c.kv[0][0])[0, 0], f(c.kv[1][0])[i, 0, :c.own_len[i]], f(c.win[0])[i, 0]])
        v = torch.cat([f(c.kv[0][1])[0, 0], f(c.kv[1][1])[i, 0, :c.own_len[i]], f(c.win[1])[i, 0]])
        x = f(c.q)[i] @ k.T * c.scale
        x[:, :, -5:].masked_fill_(torch.ones(5, 5, dtype=torch.bool, device=DEV).triu(1), -np.inf)
        p = torch.softmax(x, -1)
        err = (o[i].double() - p @ v).abs()
        assert bool((err <= 2.0 ** -8 * (p @ v.abs() + (p @ v).abs()) + 2.0 ** -13).all())
        assert float((lse[i].double() - torch.logsumexp(x, -1)).abs().max()) <= 2e-4


def ragged(n, most, seed, always=()):
    lens = torch.randint(0, most + 1, (n,), generator=I.generator(seed)).tolist()
    lens[:len(always)] = always
    return lens


PLANS = {   # b, groups, h_q, h_kv, d, w, n_prefix, n_own, page, prefix lengths, own lengths
    # more prefixes than CTAs: all on the line
    "prefixes on the line": (200, 200, 8, 1, 64, 2, 700, 100, 16, ragged(200, 700, 1, (0, 700, 1)),
                             ragged(200, 100, 2)),
    # lengths on the device: the split is searched there
    "ragged prefixes": (12, 4, 40, 8, 128, 5, 6000, 300, 64, [6000, 1, 0, 4500],
                        ragged(12, 300, 3, (0, 300))),
    "40 ragged groups": (80, 40, 4, 1, 64, 3, 3001, 64, 0, ragged(40, 3001, 4, (3001, 0)), None),
    "one long prefix among empty ones": (3, 3, 16, 2, 128, 4, 20000, 40, 0, [0, 20000, 1],
                                         [40, 0, 7]),
    # lengths known to the host, two pairs of row tiles and a single
    "pairs and a single": (16, 1, 64, 8, 128, 5, 5000, 400, 16, None, ragged(16, 400, 5, (0, 400))),
    "pairs and a single, equal lengths": (16, 1, 64, 8, 64, 5, 5000, 130, 0, None, None),
    # own parts cut over many CTAs, several row tiles of one sequence
    "a long own part": (2, 1, 8, 1, 64, 3, 0, 30000, 48, None, [30000, 17]),
    "own row tile pairs": (2, 1, 64, 1, 128, 5, 1000, 3000, 0, None, [3000, 129]),
    # three row tiles over 387 tiles: segments of one tile, the most there are
    "segments of one tile": (1, 1, 64, 1, 64, 5, 0, 49400, 0, None, None),
    "segments of one tile, ragged": (1, 1, 64, 1, 64, 5, 0, 60000, 16, None, [49400]),
    "equal own parts": (16, 2, 16, 2, 128, 1, 0, 2048, 64, None, None),
}


@pytest.mark.parametrize("plan", PLANS)
def test_plans(plan):
    """The ways the work is shared out, at sizes where CTAs hold parts of
    items, against fp64 on the GPU."""
    b, groups, hq, hkv, d, w, n_p, n_o, page, plen, olen = PLANS[plan]
    c = Case(b, groups, hq, hkv, d, w, n_p, n_o, page=page, prefix_len=plen, own_len=olen, seed=31)
    o, lse = c.run()
    f = lambda x: x.to(DEV).double()
    diagonal = torch.ones(w, w, dtype=torch.bool, device=DEV).triu(1)
    for i in range(b):
        g = i // (b // groups)
        ends = (plen[g] if plen else n_p, olen[i] if olen else n_o)
        k, v = (torch.cat([f(c.kv[0][x])[g, :, :ends[0]], f(c.kv[1][x])[i, :, :ends[1]],
                           f(c.win[x])[i]], 1).repeat_interleave(hq // hkv, 0) for x in range(2))
        x = f(c.q)[i] @ k.transpose(1, 2) * c.scale
        x[:, :, -w:].masked_fill_(diagonal, -np.inf)
        p = torch.softmax(x, -1)
        err = (o[i].double() - p @ v).abs()
        assert bool((err <= 2.0 ** -8 * (p @ v.abs() + (p @ v).abs()) + 2.0 ** -13).all()), i
        assert float((lse[i].double() - torch.logsumexp(x, -1)).abs().max()) <= 2e-4, i


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 128])
def test_tiles_of_one_box(d, page):
    """Tiles loaded as one box (contiguous caches, pages of 128): the second of
    the two load warps has no box of V, at d 64 none of K either, and must keep
    up with the ring all the same.  Many laps, short and long segments, launch
    after launch: no wait runs out, equal bits."""
    g = I.generator(d + page)
    own = torch.randint(0, 4, (24,), generator=g).mul(100).tolist()
    c = Case(24, 1, 4, 1, d, 3, 2500, 300, page=page, own_len=own, seed=d)
    long = Case(1, 1, 16, 8, d, 2, 0, 60000, page=page, win=False, seed=d + 1)
    first = c.check()
    q, a, ws = c.q.to(DEV), c.args(), c.workspace()
    lq, la, lws = long.q.to(DEV), long.args(), long.workspace()
    o, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    lo, llse = torch.empty_like(lq), torch.empty(lq.shape[:3], device=DEV)
    for _ in range(100):
        N.dustin_prefix_verify_attn(q=q, o=o, lse=lse, ws=ws, **a)
        N.dustin_prefix_verify_attn(q=lq, o=lo, lse=llse, ws=lws, **la)
    H.sync()
    assert flags() == 0
    assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    assert all(torch.equal(x, y) for x, y in zip((lo, llse), long.run()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("where", ["one row of q", "one sequence of q", "a key of the prefix",
                                   "a key of one sequence", "a key of one window"])
def test_nan_scores_stay_nan(where, page, d):
    """A row with a NaN score is NaN, o and lse, also where all its scores are
    NaN or its other parts see nothing; the other rows are what they are.  The
    shape has row tile pairs and a single, segments of one tile and of several."""
    c = Case(7, 1, 16, 2, d, 5, 900, 300, page=page, prefix_len=[897], seed=d + page,
             own_len=[300, 0, 129, 1, 257, 0, 40])
    clean = c.run()
    nan = float("nan")
    if where == "one row of q":
        c.q[2, 9, 3, 5] = nan
    elif where == "one sequence of q":
        c.q[1] = nan
    else:
        i, at, j = {"a key of the prefix": (0, 0, 600), "a key of one sequence": (4, 1, 200),
                    "a key of one window": (5, 2, 1)}[where]
        x = (c.kv + [c.win])[at][0]
        x[i, 1, j, 7] = nan
        if at == 2:
            c.dev_win[0].copy_(x)
        elif page:
            c.stored[at][0][int(c.tables[at][i, j // page]), 1, j % page, 7] = nan
        else:
            c.stored[at][0].copy_(torch.where(torch.isnan(c.stored[at][0]), c.stored[at][0],
                                              x.to(DEV)))
    o, lse = c.run()
    want_o, want_lse, spread = c.oracle()
    bad = np.isnan(want_lse)
    assert bad.any() and not bad.all()
    np.testing.assert_array_equal(np.isnan(want_o), np.broadcast_to(bad[..., None], want_o.shape))
    np.testing.assert_array_equal(np.isnan(H.f64(lse)), bad)
    np.testing.assert_array_equal(np.isnan(H.f64(o)), np.isnan(want_o))
    good = ~bad
    err = np.abs(H.f64(o) - want_o)[good]
    assert np.all(err <= (2.0 ** -8 * (spread + np.abs(want_o)) + 2.0 ** -13)[good])
    np.testing.assert_allclose(H.f64(lse)[good], want_lse[good], atol=2e-4, rtol=0)
    assert not torch.isnan(clean[0]).any() and flags() == 0


def test_nan_and_infinite_scores_of_rows_with_little_to_see():
    """A NaN in the only position a row sees, in any part; scores of -inf alone
    are as nothing seen, one of +inf is NaN."""
    for n_p, n_o, win in ((1, 0, False), (0, 1, False), (0, 0, True), (40, 3, False)):
        c = Case(3, 1, 4, 2, 64, 1, n_p, n_o, win=win, seed=n_p)
        c.q[1] = float("nan")
        o, lse = c.run()
        nan = torch.isnan(lse).cpu()
        assert nan[1].all() and not nan[[0, 2]].any()
        assert torch.isnan(o[1]).all() and not torch.isnan(o[[0, 2]]).any()
    c = Case(2, 1, 2, 1, 64, 1, 200, 3, win=False, seed=1, own_len=[0, 3])
    c.q.fill_(1.0)
    c.stored[0][0].fill_(float("-inf"))
    o, lse = c.run()                                 # sequence 1 still sees its own three
    assert not o[0].any() and torch.isneginf(lse[0]).all()
    s = (c.q[1, 0, 0].double() @ c.kv[1][0][1, 0].double().T) * c.scale
    assert abs(float(torch.logsumexp(s, -1)) - float(lse[1, 0, 0])) < 2e-4
    c.stored[0][0][0, 0, 150] = float("inf")
    o, lse = c.run()
    assert torch.isnan(o).all() and torch.isnan(lse).all()
