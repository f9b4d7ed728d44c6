"""The 4-bit cache on the GPU against its oracle.

Writing and reading are exact: every comparison is of bits.

Attention's tolerances.  K and V enter as the records stand for them.  A weight
is rounded to f16 (half a step, 2^-11 of it) and the result to bf16 (2^-8).  A
score is an fp32 sum of 64 or 128 products, whose partial sums the tensor cores may
cut off (2^-23 each): for q and k of about 1 with d^-0.5, sum |q k| scale is 8 or
less, so a score is off by 128 * 2^-23 * 8 < 2^-13, a weight and the sum of weights
each by that much of themselves (the exponential's 2^-22 beside it), O by twice
that: |error| <= 2^-8 |o| + (2^-11 + 2^-12) sum_j p_j |v_j|, element by element.
LSE: 2^-13 < 2e-4.  Where scores are larger, both go by the largest sum |q k| scale."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as Q
from sparse_kv_verification_gb300 import build, inputs as I, native as N
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
INDEX_RANGE, PAGE_RANGE = 1, 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return N.load()


def flags():
    f = ctypes.c_uint32(0)
    N.load().dustin_device_status(ctypes.byref(f))
    return f.value


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


# ---------------------------------------------------------- writing and reading

def test_every_largest_magnitude():
    """All 2^15 bf16 magnitudes as the largest of 16 channels, in turn positive and
    negative, the others anything up to it; in K and, reversed, in V."""
    r = np.random.default_rng(0)
    m = np.arange(1 << 15, dtype=np.uint16)
    others = (r.random((1 << 15, 15)) * (m[:, None] + 1)).astype(np.uint16)
    others |= r.integers(0, 2, others.shape).astype(np.uint16) << 15
    block = np.concatenate([(m | (m & 1) << 15)[:, None], others], 1)
    block = np.take_along_axis(block, r.permuted(np.tile(np.arange(16), (1 << 15, 1)), axis=1), 1)
    rows = torch.from_numpy(block.reshape(1, 1, -1, 128).view(np.int16)).view(torch.bfloat16)
    k, v = rows.to(DEV), rows.flip(2).contiguous().to(DEV)
    w = rows.shape[2]
    for exps in ((0, 0), (-40, 13)):
        cache = torch.full((1, 1, w, 144), 0xab, dtype=torch.uint8, device=DEV)
        kv4 = N.kv4_desc(cache, None, *exps)
        N.dustin_kv4_write([N.kv_desc(k, v)], [kv4], 1, 1, 128, w, w)
        want = Q.quantise(f64(k), f64(v), *exps)
        np.testing.assert_array_equal(cache.cpu().numpy(), want)
        bk, bv = torch.zeros_like(k), torch.zeros_like(v)
        N.dustin_kv4_read([kv4], [N.kv_desc(bk, bv)], 1, 1, 128, w, w)
        for got, x in zip((bk, bv), Q.dequantise(want, 128, *exps)):
            np.testing.assert_array_equal(f64(got), x)
    assert flags() == 0


def test_every_border_of_two_codes():
    """For each scale, the borders of its codes and the bf16 numbers next to them,
    in blocks whose largest magnitude gives that scale."""
    scales = Q.SCALES[1:]
    values = []
    for s in scales:
        b = torch.tensor((Q.STEPS[1:] + Q.STEPS[:-1]) / 2 * s, dtype=torch.float64).bfloat16()
        up = (b.view(torch.int16) + 1).view(torch.bfloat16)
        down = (b.view(torch.int16) - 1).view(torch.bfloat16)
        top = torch.tensor([6 * s]).bfloat16()
        for x in (b, up, down):
            values.append(torch.cat([x, -x, top, torch.zeros(1).bfloat16()]))
    rows = torch.stack(values)
    rows = torch.cat([rows, rows[:(-len(rows)) % 8]]).view(1, 1, -1, 128)
    w = rows.shape[2]
    cache = torch.zeros((1, 1, w, 144), dtype=torch.uint8, device=DEV)
    k = rows.to(DEV)
    N.dustin_kv4_write([N.kv_desc(k, k)], [N.kv4_desc(cache)], 1, 1, 128, w, w)
    np.testing.assert_array_equal(cache.cpu().numpy(), Q.quantise(f64(k), f64(k)))


class Rows:
    """bf16 rows [layers][b][h_kv][w][d] and 4-bit caches for n positions, each
    contiguous or paged (with a page outside the pool if `bad`)."""

    def __init__(self, layers, b, hkv, d, n, w, src_page, page, seed, bad=False):
        g = I.generator(seed)
        self.__dict__.update(layers=layers, b=b, hkv=hkv, d=d, n=n, w=w, page=page, src_page=src_page)
        r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
        spread = torch.exp2(torch.randint(-12, 5, (layers, b, hkv, w, d // 16), generator=g).float())
        self.rows = [r(layers, b, hkv, w, d) * spread.repeat_interleave(16, -1).bfloat16()
                     for _ in range(2)]
        self.table = self.src_table = None
        rec = Q.record_size(d)
        if page:
            per = -(-n // page)
            self.table = torch.randperm(b * per + 2, generator=g)[:b * per].int().view(b, per)
            if bad:
                self.table[0, 0], self.table[-1, -1] = -1, b * per + 2
            shape = (b * per + 2, hkv, page, rec)
        else:
            shape = (b, hkv, n, rec)
        self.caches = [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).to(DEV)
                       for _ in range(layers)]
        if src_page:
            per = -(-w // src_page)
            self.src_table = torch.randperm(b * per, generator=g).int().view(b, per)

    def src(self, x):
        """Layer x's K and V rows as tensors on the GPU, laid out as the case asks."""
        out = []
        for t in self.rows:
            t = t[x]
            if not self.src_page:
                # Heads and positions the other way round in memory.
                out.append(t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2))
                continue
            per = self.src_table.shape[1]
            pool = torch.zeros((self.b * per, self.hkv, self.src_page, self.d), dtype=torch.bfloat16)
            padded = torch.zeros((self.b, self.hkv, per * self.src_page, self.d), dtype=torch.bfloat16)
            padded[:, :, :self.w] = t
            pool[self.src_table.long()] = padded.view(self.b, self.hkv, per, self.src_page, self.d) \
                .transpose(1, 2)
            out.append(pool.to(DEV))
        return out

    def kv4(self, k_exp=0, v_exp=0):
        t = None if self.table is None else self.table.to(DEV)
        self.dev_table = t                               # kept alive with the descriptors
        return [N.kv4_desc(c, t, k_exp, v_exp) for c in self.caches]

    def place(self, cache, i, j):
        """Records [h_kv][record] of position j of sequence i; None: no page."""
        if self.table is None:
            return cache[i, :, j]
        p = int(self.table[i, j // self.page])
        return cache[p, :, j % self.page] if 0 <= p < len(cache) else None


SHAPES = [(1, 1, 1, 64, 16, 1, 0, 0), (1, 1, 1, 128, 16, 1, 0, 16), (2, 3, 2, 64, 100, 37, 0, 16),
          (2, 3, 2, 128, 100, 37, 16, 48), (3, 2, 4, 128, 33, 33, 0, 0), (130, 1, 1, 64, 20, 3, 0, 16),
          (1, 17, 5, 128, 64, 5, 32, 64), (1, 5, 1, 64, 1000, 700, 0, 0)]


@pytest.mark.parametrize("layers,b,hkv,d,n,w,src_page,page", SHAPES)
@pytest.mark.parametrize("ragged", [False, True])
def test_rows_are_written_and_read_back(layers, b, hkv, d, n, w, src_page, page, ragged):
    c = Rows(layers, b, hkv, d, n, w, src_page, page, seed=n + w + b)
    g = I.generator(b)
    start = torch.randint(0, n - w + 1, (b,), generator=g).tolist() if ragged or n > w else None
    lens = (torch.randint(-1, w + 2, (b,), generator=g)).tolist() if ragged else None
    src = [c.src(x) for x in range(layers)]
    st = None if c.src_table is None else c.src_table.to(DEV)
    before = [x.cpu().numpy().copy() for x in c.caches]
    kv4 = c.kv4(-3, 2)
    N.dustin_kv4_write([N.kv_desc(*s, st) for s in src], kv4, b, hkv, d, n, w, start=i32(start),
                       w_len=i32(lens))
    idx = [[(start[i] if start else 0) + t for t in range(w)] for i in range(b)]
    back = [[torch.full((b, hkv, w, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            for _ in range(layers)]
    N.dustin_kv4_read(kv4, [N.kv_desc(*x) for x in back], b, hkv, d, n, w, idx=i32(idx),
                      k_len=i32(lens))
    for x in range(layers):
        want = before[x].copy()
        for i in range(b):
            m = w if lens is None else min(max(lens[i], 0), w)
            rec = Q.quantise(*(f64(t[x, i, :, :m]) for t in c.rows), -3, 2)
            for t in range(m):
                c.place(want, i, idx[i][t])[:] = rec[:, t]
            for got, y in zip(back[x], Q.dequantise(rec, d, -3, 2)):
                np.testing.assert_array_equal(f64(got[i, :, :m]), y)
                assert (got[i, :, m:] == 7.0).all()
        np.testing.assert_array_equal(c.caches[x].cpu().numpy(), want)   # the rest as it was
    assert flags() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_positions_and_pages_out_of_range_are_left_out(d):
    b, hkv, n, w, page = 3, 2, 64, 20, 16
    c = Rows(1, b, hkv, d, n, w, 0, page, seed=d, bad=True)
    before = c.caches[0].cpu().numpy().copy()
    start = [0, 50, -5]
    big = [2 ** 31 - 1, -2 ** 31, 64]
    src = c.src(0)
    for st, flag in ((start, INDEX_RANGE | PAGE_RANGE), (big, INDEX_RANGE)):
        N.dustin_kv4_write([N.kv_desc(*src)], c.kv4(), b, hkv, d, n, w, start=i32(st))
        assert flags() == flag
    want = before.copy()
    rec = Q.quantise(*(f64(t[0]) for t in c.rows))
    for i in range(b):
        for t in range(w):
            to = c.place(want, i, start[i] + t) if 0 <= start[i] + t < n else None
            if to is not None:
                to[:] = rec[i, :, t]
    np.testing.assert_array_equal(c.caches[0].cpu().numpy(), want)
    idx = [[0, 17, 5, -1, 63], [64, 2 ** 31 - 1, -2 ** 31, 3, 3], [63, 48, 1, 0, 47]]
    back = [torch.full((b, hkv, 5, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    N.dustin_kv4_read(c.kv4(), [N.kv_desc(*back)], b, hkv, d, n, 5, idx=i32(idx))
    assert flags() == INDEX_RANGE | PAGE_RANGE
    for i in range(b):
        for t, j in enumerate(idx[i]):
            r = c.place(want, i, j) if 0 <= j < n else None
            for got, part in zip(back, (0, 1)):
                x = np.full((hkv, d), 7.0) if r is None else Q.dequantise(r, d)[part]
                np.testing.assert_array_equal(f64(got[i, :, t]), x)


def test_a_cache_past_four_gigabytes():
    n, w = 31_000_000, 3
    cache = torch.empty((1, 1, n, 144), dtype=torch.uint8, device=DEV)   # 4.5 GB
    k, v = (torch.randn((1, 1, w, 128), generator=I.generator(s)).bfloat16().to(DEV) for s in (1, 2))
    kv4 = N.kv4_desc(cache)
    N.dustin_kv4_write([N.kv_desc(k, v)], [kv4], 1, 1, 128, n, w, start=i32([n - w]))
    want = Q.quantise(f64(k), f64(v))
    np.testing.assert_array_equal(cache[:, :, n - w:].cpu().numpy(), want)
    back = [torch.zeros_like(k) for _ in range(2)]
    at = i32([[n - w, n - 2, n - 1]])
    N.dustin_kv4_read([kv4], [N.kv_desc(*back)], 1, 1, 128, n, w, idx=at)
    rk, rv = Q.dequantise(want, 128)
    np.testing.assert_array_equal(f64(back[0]), rk)
    np.testing.assert_array_equal(f64(back[1]), rv)
    q = torch.randn((1, 2, 1, 128), generator=I.generator(3)).bfloat16()
    o, lse = torch.empty_like(q, device=DEV), torch.empty((1, 2, 1), device=DEV)
    ws = N.workspace(N.dustin_kv4_verify_attn_workspace_size(1, 2, 1, 128, 1, w), DEV)
    N.dustin_kv4_verify_attn(q.to(DEV), kv4, 1, n, w, 0.1, o, lse, ws, idx=at)
    check(o, lse, Q.attention(f64(q), rk, rv, 0.1, [np.arange(w)]))
    assert flags() == 0


def test_calls_without_work():
    cache = torch.zeros((2, 1, 4, 144), dtype=torch.uint8, device=DEV)
    rows = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16, device=DEV)
    kv4, kv = N.kv4_desc(cache), N.kv_desc(rows, rows)
    before = N.dustin_launch_count()
    for w in (0, 4):
        N.dustin_kv4_write([], [], 2, 1, 128, 4, w)
        N.dustin_kv4_read([], [], 2, 1, 128, 4, w)
    N.dustin_kv4_write([kv], [kv4], 2, 1, 128, 4, 0)
    N.dustin_kv4_read([kv4], [kv], 2, 1, 128, 4, 0)
    assert N.dustin_launch_count() == before


# ------------------------------------------------------------------- attention

def check(o, lse, want, large=1.0):
    """Within the tolerances above; `large`: sum |q k| scale in units of 8."""
    ro, rl, spread = want
    o, lse = f64(o), f64(lse)
    nan = np.isnan(rl)
    np.testing.assert_array_equal(np.isnan(lse), nan)
    np.testing.assert_array_equal(np.isnan(o), np.broadcast_to(nan[..., None], o.shape))
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(lse[fin] - rl[fin]) <= 2e-4 * large)
    assert not o[np.isneginf(rl)].any()
    bound = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -12 * large) * spread
    assert np.all(np.abs(o[fin] - ro[fin]) <= bound[fin])


class Case:
    """Inputs on the CPU; records on the GPU, all bytes that no position owns 0xff
    (codes -6, scales NaN)."""

    def __init__(self, b, hq, hkv, d, w, n, k=None, page=0, win=True, k_len=None, idx=None, seed=0,
                 k_exp=0, v_exp=0, layout="rows"):
        g = I.generator(seed)
        r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
        self.__dict__.update(b=b, hkv=hkv, d=d, n=n, page=page, k_len=k_len, scale=d ** -0.5,
                             exps=(k_exp, v_exp), layout=layout)
        self.q = r(b, hq, w, d)
        self.rec = Q.quantise(f64(r(b, hkv, n, d)) * 2.0 ** k_exp, f64(r(b, hkv, n, d)) * 2.0 ** v_exp,
                              k_exp, v_exp)
        if idx == "some":                                # ascending, as a selection gives them
            k = n // 3 if k is None else k
            idx = torch.stack([torch.randperm(n, generator=g)[:k].sort().values for _ in range(b)])
        elif idx == "any":                               # any order, repeats
            k = n // 2 if k is None else k
            idx = torch.randint(0, n, (b, k), generator=g)
        self.idx = None if idx is None else idx.tolist()
        self.k = n if k is None else k
        self.win = [r(b, hkv, w, d), r(b, hkv, w, d)] if win else None
        if page:
            per = -(-n // page)
            perm = torch.randperm(b * per + 3, generator=g).int()
            self.table = perm[:b * per].view(b, per)

    def upload(self):
        rec = torch.from_numpy(self.rec)
        b, hkv, n, size = rec.shape
        used = torch.zeros((b, n), dtype=torch.bool)
        for i, at in enumerate(self.seen()):
            used[i, torch.as_tensor(at, dtype=torch.long)] = True
        rec = torch.where(used[:, None, :, None], rec, torch.tensor(0xff, dtype=torch.uint8))
        t = None
        if self.page:
            per = self.table.shape[1]
            padded = torch.full((b, hkv, per * self.page, size), 0xff, dtype=torch.uint8)
            padded[:, :, :n] = rec
            cache = torch.full((b * per + 3, hkv, self.page, size), 0xff, dtype=torch.uint8)
            ok = (self.table >= 0) & (self.table < len(cache))
            pages = padded.view(b, hkv, per, self.page, size).transpose(1, 2)
            cache[self.table[ok].long()] = pages[ok]
            t = self.table.to(DEV)
        else:
            cache = rec
        if self.layout == "positions":                   # [..][position][h_kv][record]
            cache = cache.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
        elif self.layout == "spread":                    # records 160 or 96 bytes apart
            wide = torch.full((*cache.shape[:3], size + 16), 0xff, dtype=torch.uint8)
            wide[..., :size] = cache
            cache = wide.to(DEV)[..., :size]
        else:
            cache = cache.to(DEV)
        self.kept = (cache, t)
        return N.kv4_desc(cache, t, *self.exps)

    def seen(self):
        out = []
        for i in range(self.b):
            m = self.k if self.k_len is None else min(max(self.k_len[i], 0), self.k)
            at = np.arange(m) if self.idx is None else np.array(self.idx[i][:m], dtype=np.int64)
            at = at[(at >= 0) & (at < self.n)]
            if self.page:
                p = self.table[i, torch.from_numpy(at // self.page)].numpy()
                at = at[(p >= 0) & (p < self.b * self.table.shape[1] + 3)]
            out.append(at)
        return out

    def run(self, kv=None, ws=None, stream=None):
        q = self.q.to(DEV)
        b, hq, w, d = q.shape
        o = torch.full_like(q, float("nan"))
        lse = torch.full((b, hq, w), float("nan"), device=DEV)
        if ws is None:
            ws = N.workspace(N.dustin_kv4_verify_attn_workspace_size(b, hq, self.hkv, d, w, self.k),
                             DEV).fill_(255)
        self.dev_win = None if self.win is None else [x.to(DEV) for x in self.win]
        N.dustin_kv4_verify_attn(q, kv or self.upload(), self.hkv, self.n, self.k, self.scale, o, lse,
                                 ws, idx=i32(self.idx), k_len=i32(self.k_len),
                                 win=None if self.win is None else N.kv_desc(*self.dev_win))
        H.sync()
        return o, lse

    def oracle(self):
        k, v = Q.dequantise(self.rec, self.d, *self.exps)
        win = [None, None] if self.win is None else [f64(x) for x in self.win]
        return Q.attention(f64(self.q), k, v, self.scale, self.seen(), *win)

    def check(self, large=1.0):
        o, lse = self.run()
        check(o, lse, self.oracle(), large)
        return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 300])
@pytest.mark.parametrize("page", [0, 16])
def test_lengths_around_a_tile(n, page, d):
    Case(1, 4, 2, d, 1, n, page=page, win=False, seed=n).check()
    Case(2, 4, 2, d, 3, n, page=page, seed=n).check()
    assert flags() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,w", [(1, 1, 1), (16, 1, 1), (17, 1, 1), (8, 1, 4), (33, 1, 1), (40, 2, 2),
                                      (48, 1, 1), (8, 1, 7), (64, 8, 8), (13, 1, 5), (8, 1, 16), (6, 3, 50)])
def test_numbers_of_query_rows(hq, hkv, w, d):
    """1 to 128 rows of a kv head: every padding, one block of rows and two."""
    Case(2, hq, hkv, d, w, 200, seed=hq + w).check()
    Case(1, hq, hkv, d, w, 150, idx="any", page=16, win=False, seed=hq * w).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 32, 48, 64, 128, 192])
@pytest.mark.parametrize("idx", [None, "some", "any"])
def test_ragged_batches(idx, page, d):
    """Empty sequences, lengths past both ends, pages that end inside a tile."""
    lens = [0, 700, 1, 128, -3, 900, 257, 16]
    Case(8, 10, 2, d, 2, 700, k=640 if idx else None, page=page, k_len=lens, idx=idx, seed=page).check()
    Case(8, 4, 1, d, 1, 700, k=640 if idx else None, page=page, k_len=lens, idx=idx, win=False,
         seed=page).check()
    assert flags() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["positions", "spread"])
@pytest.mark.parametrize("page", [0, 48])
def test_other_layouts(page, layout, d):
    Case(3, 8, 4, d, 3, 333, page=page, layout=layout, k_len=[333, 40, 0], seed=d).check()
    Case(3, 8, 4, d, 3, 333, page=page, layout=layout, idx="some", seed=d).check()


def test_nothing_to_see():
    for win in (False, True):
        Case(2, 4, 2, 64, 3, 0, win=win).check()
        Case(2, 4, 2, 128, 3, 50, k=0, idx="any", win=win).check()
        Case(3, 4, 2, 128, 3, 50, k_len=[0, 0, 0], win=win).check()
    c = Case(2, 4, 2, 64, 1, 0, win=False)
    o, lse = torch.ones((2, 4, 1, 64), dtype=torch.bfloat16, device=DEV), torch.ones((2, 4, 1), device=DEV)
    ws = N.workspace(N.dustin_kv4_verify_attn_workspace_size(2, 4, 2, 64, 1, 0), DEV)
    N.dustin_kv4_verify_attn(c.q.to(DEV), None, 2, 0, 0, 0.1, o, lse, ws)      # no cache at all
    assert not o.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("idx", [None, "any"])
@pytest.mark.parametrize("n,rows", [(40000, 1), (57000, 5), (9000, 3)])
def test_equal_calls_give_equal_bits(d, n, rows, idx):
    """A few tiles per SM, taken while the code is still being fetched: the warps of
    K, V and the softmax are then the furthest apart."""
    c = Case(1, 8, 1, d, rows, n, idx=idx, win=False, seed=n)
    o, lse = c.check()
    for _ in range(40):
        again = c.run()
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("b,hkv,n,lens", [(300, 2, 130, None), (1, 1, 40000, None), (3, 2, 5000, None),
                                          (90, 1, 600, "ragged"), (2, 4, 9000, [8999, 1])])
def test_shares_of_the_line(b, hkv, n, lens):
    """More units than SMs, one unit shared by all of them, segments that begin and
    end inside a unit."""
    if lens == "ragged":
        lens = torch.randint(0, n + 1, (b,), generator=I.generator(b)).tolist()
    c = Case(b, 4 * hkv, hkv, 64, 1, n, k_len=lens, win=False, seed=b)
    o, lse = c.check()
    again = c.run()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])             # a fixed order


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("idx", [None, "some"])
def test_exponents(idx, d):
    for k_exp, v_exp in ((5, -7), (-6, 4), (-64, 64)):
        c = Case(2, 8, 2, d, 2, 260, idx=idx, k_exp=k_exp, v_exp=v_exp, seed=3)
        c.scale *= 2.0 ** -k_exp
        c.win = [c.win[0] * 2.0 ** k_exp, c.win[1] * 2.0 ** v_exp]
        c.check()


@pytest.mark.parametrize("by", [2.0 ** -100, 2.0 ** -20, 2.0 ** 15, 2.0 ** 60])
def test_queries_of_any_size(by):
    """q past f16's range at either end; entries far below their row's largest."""
    c = Case(2, 8, 2, 128, 2, 260, seed=5)
    c.q = c.q * by
    c.scale /= by
    c.check()
    c.q[:, :, :, ::3] *= 2.0 ** -30
    c.check()


def test_scores_that_grow_and_fall():
    """References that move in every tile, in some rows only, and stay behind."""
    b, hq, d, n = 2, 8, 128, 1500
    for sign in (1, -1):
        c = Case(b, hq, 1, d, 1, n, seed=6)
        k, v = Q.dequantise(c.rec, d)
        ramp = sign * np.linspace(-1, 1, n)[None, None, :, None]
        lean = f64(c.q[:, :1, 0]) / np.linalg.norm(f64(c.q[:, :1, 0]), axis=-1, keepdims=True)
        c.rec = Q.quantise(k + 100 * ramp * lean[:, :, None], v)
        # Scores of up to 100: sum |q k| scale is below 160.
        c.check(large=20)


def test_huge_scores_stay_finite_weights():
    """Differences of scores beyond every exponent: the largest takes all."""
    c = Case(2, 4, 1, 64, 2, 400, win=False, seed=7)
    c.scale = 1e6
    o, lse = c.run()
    k, v = Q.dequantise(c.rec, 64)
    s = np.einsum("bhtd,bnd->bhtn", f64(c.q), k[:, 0]) * 1e6
    best = s.argmax(-1)
    gap = np.sort(s, -1)
    clear = gap[..., -1] - gap[..., -2] > 100                # beyond fp32's rounding of 1e7
    assert clear.any()
    for i, h, t in zip(*np.nonzero(clear)):
        np.testing.assert_allclose(f64(o)[i, h, t], v[i, 0, best[i, h, t]], rtol=2.0 ** -7, atol=0)
    np.testing.assert_allclose(f64(lse), s.max(-1), rtol=1e-5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("idx", [None, "some"])
@pytest.mark.parametrize("where", ["a row of q", "a sequence of q", "a key", "a value", "a window key"])
def test_nan_stays_where_it_is(where, idx, d):
    c = Case(3, 12, 2, d, 3, 400, idx=idx, k_len=[133, 90, 0], seed=d)
    if where == "a row of q":
        c.q[0, 7, 1, 5] = float("nan")
    elif where == "a sequence of q":
        c.q[1] = float("nan")
    elif where == "a window key":
        c.win[0][2, 1, 1, 7] = float("nan")
    else:
        j = 60 if idx is None else c.idx[0][60]
        c.rec[0, 1, j, d + (2 if where == "a key" else d // 16 + 2)] = 0x7f
    o, lse = c.run()
    want = c.oracle()
    if where == "a value":                                   # 16 channels of the rows that see it
        bad = np.isnan(want[0])
        assert bad.any() and not bad.all()
        np.testing.assert_array_equal(np.isnan(f64(o)), bad)
        assert np.all(np.abs(f64(lse) - want[1])[np.isfinite(want[1])] <= 2e-4)
        bound = 2.0 ** -8 * np.abs(want[0]) + (2.0 ** -11 + 2.0 ** -12) * want[2]
        assert np.all((np.abs(f64(o) - want[0]) <= bound)[~bad])
    else:
        check(o, lse, want)
        assert np.isnan(want[1]).any() and not np.isnan(want[1]).all()
    assert flags() == 0


def test_infinite_queries():
    """Scores of +inf are NaN; of -inf alone, nothing seen."""
    c = Case(2, 4, 2, 64, 2, 300, win=False, seed=2)
    c.rec[:, :, :, :2] = 0x22                                # K channels 0 .. 3 are positive
    c.q[0, 1, 0, 0] = float("inf")
    c.q[1, 3, 1, 1] = float("-inf")
    o, lse = c.check()
    assert torch.isnan(lse[0, 1, 0]) and torch.isneginf(lse[1, 3, 1])


@pytest.mark.parametrize("d", [64, 128])
def test_indices_and_pages_out_of_range_are_left_out(d):
    c = Case(3, 4, 2, d, 2, 300, idx="any", k=200, seed=d)
    for i, at, to in ((0, 0, -1), (0, 63, 300), (0, 64, 2 ** 31 - 1), (1, 130, -2 ** 31)):
        c.idx[i][at] = to
    c.idx[2] = [300] * 200                                   # nothing left but the window
    c.check()
    assert flags() == INDEX_RANGE
    for page in (16, 48):
        for idx in (None, "some"):
            c = Case(3, 4, 2, d, 2, 500, page=page, idx=idx, seed=page)
            c.table[0, 0] = -1
            c.table[1, 3:] = 3 * c.table.shape[1] + 3
            c.table[2] = 1 << 30
            c.check()
            assert flags() == PAGE_RANGE
            c.win = None
            c.check()
            assert flags() == PAGE_RANGE


def test_streams_workspaces_and_graphs():
    """Two calls at once on two streams with a workspace each, and two captured
    graphs replayed beside one another, give the bits of a call alone."""
    cases = [Case(4, 8, 2, 128, 4, 2000, idx="some", k=900, seed=1),
             Case(2, 40, 8, 64, 1, 3000, page=16, k_len=[2900, 17], win=False, seed=2)]
    alone = [c.run() for c in cases]
    side = [torch.cuda.Stream() for _ in cases]
    made = []
    for c, st in zip(cases, side):
        kv, q = c.upload(), c.q.to(DEV)
        o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device=DEV)
        ws = N.workspace(N.dustin_kv4_verify_attn_workspace_size(
            c.b, q.shape[1], c.hkv, c.d, q.shape[2], c.k), DEV)
        c.dev_win = None if c.win is None else [x.to(DEV) for x in c.win]
        idx, lens = i32(c.idx), i32(c.k_len)

        def call(stream, c=c, kv=kv, q=q, o=o, lse=lse, ws=ws, idx=idx, lens=lens):
            N.dustin_kv4_verify_attn(q, kv, c.hkv, c.n, c.k, c.scale, o, lse, ws, idx=idx, k_len=lens,
                                     win=None if c.win is None else N.kv_desc(*c.dev_win), stream=stream)
        made.append((call, o, lse))
    H.sync()
    for _ in range(3):
        for (call, _, _), st in zip(made, side):
            call(st)
    H.sync()
    for (_, o, lse), want in zip(made, alone):
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        o.zero_(), lse.zero_()
    graphs = []
    for (call, _, _), st in zip(made, side):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            call(None)
            call(None)
    H.sync()
    for _ in range(3):
        for graph, st in zip(graphs, side):
            with torch.cuda.stream(st):
                graph.replay()
    H.sync()
    for (_, o, lse), want in zip(made, alone):
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert flags() == 0


@pytest.mark.parametrize("idx", [None, "some"])
@pytest.mark.parametrize("sign", [1, -1])
def test_weights_stay_finite_where_scores_are_far_apart_in_fp32(sign, idx):
    """Row maxima of either sign up to 2^29 and more (log2 units), where 8 is half of
    what neighbouring fp32 numbers are apart, or less: no weight leaves f16, and the
    largest score takes all.  A score is off by 128 * 2^-23 of sum |q k| scale, here less
    than four times the score: by less than 2^-14 of it; a gap of 10^-4 is clear."""
    c = Case(4, 8, 1, 64, 2, 900, idx=idx, win=False, seed=17)
    c.rec[:, :, :, 0] = 0x22                                 # K channels 0, 1 are positive
    c.q[..., 0] = 512.0 * sign
    k, v = Q.dequantise(c.rec, 64)
    clear = ties = 0
    for scale in np.geomspace(2e5, 6e6, 14):
        c.scale = float(np.float32(scale))
        o, lse = (f64(x) for x in c.run())
        assert np.isfinite(o).all() and np.isfinite(lse).all()
        for i, at in enumerate(c.seen()):
            s = np.einsum("htd,nd->htn", f64(c.q[i]), k[i, 0, at]) * c.scale
            best, order = s.argmax(-1), np.sort(s, -1)
            assert (order[..., -1] * sign > 0).all()
            ties += (np.abs(order[..., -1]) * np.log2(np.e) // 2 ** 27 == 1).sum()
            np.testing.assert_allclose(lse[i], order[..., -1], rtol=1e-4)
            gap = order[..., -1] - order[..., -2] > 1e-4 * np.abs(order[..., -1])
            for h, t in zip(*np.nonzero(gap)):
                np.testing.assert_allclose(o[i, h, t], v[i, 0, at[best[h, t]]], rtol=2.0 ** -8, atol=0)
                clear += 1
    assert clear > 500 and ties > 100
    assert flags() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("idx", [None, "first"])
def test_tiles_without_a_finite_score_before_others(idx, d):
    """Scores of -6 * 2^126 are beyond fp32 and so -inf, those of -0.25 * 2^126 are not: a
    row that meets only the first in a segment's first tiles sees the others all the same,
    beside rows that have finite scores everywhere; and a row that sees none is empty."""
    b, hkv, n = 76, 2, 1024                                  # eight tiles a unit, one unit a CTA of 152
    c = Case(b, 6 * hkv, hkv, d, 1, n, win=False, seed=d,
             idx=None if idx is None else torch.arange(n).expand(b, n))
    c.scale = 2.0 ** 126
    far = torch.arange(n).view(1, n) < torch.arange(b).view(b, 1) % 7 * 128 + 128
    far[3] = True                                            # nothing else
    far = far.numpy()[:, None].repeat(hkv, 1)
    c.rec[..., 0] = np.where(far, 0xf, 0x9)                  # K channels 0, 1: code -6 or -0.5, and 0
    c.rec[..., d] = np.where(far, 0x38, 0x30)                # of scale 1 or 0.5
    c.q = c.q * 2.0 ** -128
    c.q[:, ::2] = 0
    c.q[:, ::2, :, 0] = 1.0                                  # every other row: the score is K's channel 0
    o, lse = c.run()
    ro, rl, spread = c.oracle()
    none = np.broadcast_to((far.all(-1).repeat(6, 1) & (np.arange(6 * hkv) % 2 == 0))[..., None], rl.shape)
    ro[none], rl[none] = 0, -np.inf
    with np.errstate(invalid="ignore"):
        large = rl < -1e30                                   # held to 2^-20 of themselves
    assert none.sum() == 6 and large.sum() == 6 * b
    got, finite = f64(lse), large & ~none
    np.testing.assert_allclose(got[finite], rl[finite], rtol=2.0 ** -20)
    fill = torch.from_numpy(np.where(finite, rl, got))
    check(o, fill, (ro, rl, spread))
    assert flags() == 0


@pytest.mark.parametrize("idx", [None, "first"])
def test_scores_past_fp32_are_infinite(idx):
    """6 * 2^126 in the first tile, in a later one or in the last position of all: NaN, for
    the rows that meet it only."""
    b, n = 152, 1024                                         # eight tiles a unit, one unit a CTA of 152
    c = Case(b, 4, 1, 64, 1, n, win=False, seed=8, idx=None if idx is None else torch.arange(n).expand(b, n))
    c.scale = 2.0 ** 126
    c.rec[..., 0], c.rec[..., 64] = 0x09, 0x30               # K channels 0, 1: -0.25 and 0
    at = [0, 100, 300, 600, 1023, None]
    for i in range(b):
        if at[i % 6] is not None:
            c.rec[i, 0, at[i % 6], 0], c.rec[i, 0, at[i % 6], 64] = 0x07, 0x38   # 6
    c.q = c.q * 2.0 ** -128
    c.q[:, ::2] = 0
    c.q[:, ::2, :, 0] = 1.0
    o, lse = (f64(x) for x in c.run())
    want = np.zeros(lse.shape, bool)
    want[np.arange(b) % 6 != 5, ::2] = True
    np.testing.assert_array_equal(np.isnan(lse), want)
    np.testing.assert_array_equal(np.isnan(o), np.broadcast_to(want[..., None], o.shape))
    assert np.isfinite(lse[~want]).all() and flags() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("idx", [None, "some"])
@pytest.mark.parametrize("scale,k_exp,q_exp", [(2.0 ** 127.9, -64, -66), (3 * 2.0 ** -149, 64, 81),
                                               (2.0 ** -149, 64, 83)])
def test_scales_at_the_ends_of_fp32(scale, k_exp, q_exp, idx, d):
    """scale * log2 e is no fp32 number, or one of few bits, while scale * 2^k_exp and the
    scores are ordinary; and no cache at all, where a window alone meets the scale."""
    c = Case(2, 8, 2, d, 2, 260, idx=idx, win=scale > 1, k_exp=k_exp, seed=9)
    c.scale = float(np.float32(scale))
    c.q = c.q * 2.0 ** q_exp                                 # |q| scale 2^k_exp is 1/4 or so
    if c.win:
        c.win[0] = c.win[0] * 2.0 ** k_exp
    c.check(large=4)
    if c.win:
        c.k, c.idx = 0, None
        c.check(large=4)
    assert flags() == 0


@pytest.mark.parametrize("k", [0, 200])
def test_huge_scores_of_the_window(k):
    """Scores of a window from 2^20 to past 2^100 (log2 units): the largest takes all, alone and
    beside a cache."""
    c = Case(4, 8, 1, 64, 12, 200, k=k, seed=23)
    c.win[0] = c.win[0] * 4                                  # the window has the largest scores, mostly
    keys, values = Q.dequantise(c.rec, 64)
    clear = 0
    for scale in np.geomspace(1e4, 1e32, 30):
        c.scale = float(np.float32(scale))
        o, lse = (f64(x) for x in c.run())
        assert np.isfinite(o).all() and np.isfinite(lse).all()
        for i in range(4):
            for t in range(12):
                a = np.concatenate([keys[i, 0, :k], f64(c.win[0][i, 0, :t + 1])])
                v = np.concatenate([values[i, 0, :k], f64(c.win[1][i, 0, :t + 1])])
                s = f64(c.q[i, :, t]) @ a.T * c.scale
                size = (np.abs(f64(c.q[i, :, t])) @ np.abs(a).T).max(-1) * c.scale
                order = np.sort(np.concatenate([s, np.full((8, 1), -np.inf)], -1), -1)
                assert np.all(np.abs(lse[i, :, t] - order[:, -1]) <= 2.0 ** -14 * size + 6)
                # Off by 128 * 2^-23 of sum |q k| scale at most.
                for h in np.nonzero(order[:, -1] - order[:, -2] > 2.0 ** -13 * size + 100)[0]:
                    np.testing.assert_allclose(o[i, h, t], v[s[h].argmax()], rtol=2.0 ** -8, atol=1e-25)
                    clear += 1
    assert clear > 5000
    assert flags() == 0
