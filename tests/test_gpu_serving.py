"""The serving operators on the GPU against their oracle: drafted tokens,
cache compaction, shared pages.  Their results are whole numbers and moved
rows: every comparison is exact."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from sparse_kv_verification_gb300 import build, inputs as I, native as N
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
INDEX_RANGE, PAGE_RANGE, NO_PAGES, INDEX_ORDER = 1, 2, 8, 16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return N.load()


def flags():
    """Reads and clears the device flags."""
    import ctypes
    f = ctypes.c_uint32(0)
    N.load().dustin_device_status(ctypes.byref(f))
    return f.value


# ------------------------------------------------------------- drafted tokens

def token_inputs(b, w, vocab, dtype, seed, sharp=2.0):
    g = I.generator(seed)
    logits = sharp * torch.randn((b, w, vocab), generator=g)
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :w - 1] + torch.randn((b, w - 1, vocab), generator=g), -1).to(dtype)
    draft = torch.zeros((b, w - 1), dtype=torch.int32)
    if w > 1:
        draft = torch.multinomial(q.float().view(-1, vocab), 1, generator=g).view(b, w - 1).int()
    return (p, q, draft, torch.rand((b, w - 1), generator=g), torch.rand((b,), generator=g),
            torch.randint(0, w, (b,), generator=g).int())


def run_tokens(p, q, draft, ua, us, n_draft):
    b, w = p.shape[:2]
    tok = torch.full((b, w), -7, dtype=torch.int32, device=DEV)
    acc = torch.full((b,), -7, dtype=torch.int32, device=DEV)
    to = lambda t: None if t is None else t.to(DEV)
    N.dustin_verify_tokens(to(p), to(q), to(draft), to(ua), to(us), tok, acc, n_draft=to(n_draft))
    H.sync()
    return tok.cpu().numpy(), acc.cpu().numpy()


def check_tokens(p, q, draft, ua, us, n_draft):
    got = run_tokens(p, q, draft, ua, us, n_draft)
    f = lambda t: None if t is None else t.double().numpy()
    want = S.verify_tokens(f(p), f(q), draft.numpy(), None if n_draft is None else n_draft.numpy(),
                           f(ua), f(us))
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[0], want[0])
    return got


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,w,vocab", [(1, 1, 1), (1, 2, 7), (3, 4, 129), (2, 40, 1000),
                                       (1, 4, 32000), (5, 3, 50257), (40, 2, 4099),
                                       (300, 2, 257), (2, 5, 152064)])
def test_tokens_parity(b, w, vocab, dtype, ragged, drafted):
    p, q, draft, ua, us, nd = token_inputs(b, w, vocab, dtype, seed=b + w + vocab)
    check_tokens(p, q if drafted else None, draft, ua, us, nd if ragged else None)


def test_tokens_flat_row_hits_every_border():
    """A flat distribution with u on and next to the borders j / V: C_j > u
    holds first at j for u = j / V exactly, and at j - 1 just below."""
    vocab = 4096                                     # C_j = (j + 1) / V is exact
    js = torch.arange(1, vocab, 37)
    us = torch.cat([js / vocab, torch.nextafter(js / vocab, torch.zeros(1))]).float()
    p = torch.full((1, 1, vocab), 1.0 / vocab).expand(len(us), 1, vocab).contiguous()
    none = torch.zeros((len(us), 0))
    tok, _ = check_tokens(p, None, none.int(), none, us, None)
    assert tok[:len(js), 0].tolist() == js.tolist()
    assert tok[len(js):, 0].tolist() == (js - 1).tolist()


def test_tokens_edges():
    """Rows without mass, residuals without mass, one-hot rows, u at 0, 1 and
    NaN, entries that do not count, drafts outside the vocabulary."""
    vocab, nan, inf = 70, float("nan"), float("inf")
    p = torch.zeros((9, 3, vocab))
    q = torch.zeros((9, 2, vocab))
    draft = torch.zeros((9, 2), dtype=torch.int32)
    ua = torch.full((9, 2), 0.5)
    us = torch.full((9,), 0.5)
    p[1, :, 69] = q[1, :, 69] = 1.0                  # one-hot, accepted throughout
    draft[1] = 69
    p[2, :, :2] = q[2, :, :2] = 0.5                  # equal rows, u = 1: empty residual
    ua[2] = 1.0
    p[3, :, 1:4] = 0.25                              # nothing drawn where p < q
    q[3, :, :2] = 0.5
    p[4, :, 5:9] = 0.25
    us[4] = 1.0
    p[5, :, 5:9] = 0.25
    us[5] = nan
    p[6, :, 3] = 0.5
    p[6, :, 4], p[6, :, 5], p[6, :, 6] = nan, inf, -1.0
    p[7, :, 5:9] = 0.25
    ua[7] = nan
    draft[7] = 5
    q[7, :, 5] = 1.0
    p[8, :, 10] = 1.0
    draft[8, 0] = vocab                              # left out and flagged
    tok, acc = check_tokens(p, q, draft, ua, us, None)
    assert flags() == INDEX_RANGE
    assert tok[0].tolist() == [-1, -1, -1]
    assert tok[1].tolist() == [69, 69, 69] and acc[1] == 2
    assert tok[2, 0] == 1 and acc[2] == 0
    assert tok[4, 0] == 8 and tok[5, 0] == 5 and tok[6, 0] == 3 and tok[7, 0] in (6, 7)
    assert tok[8, 0] == 10
    draft[8, 0] = -1
    check_tokens(p, None, draft, ua, us, None)
    assert flags() == INDEX_RANGE


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_strided_rows(dtype):
    """Rows cut out of padded, oddly placed logits buffers, on a side stream."""
    b, w, vocab = 3, 4, 1001
    p, q, draft, ua, us, nd = token_inputs(b, w, vocab, dtype, seed=5)
    wide_p = torch.full((b, w + 1, vocab + 37), float("nan"), dtype=dtype, device=DEV)
    wide_q = torch.full((b, w, vocab + 12), float("nan"), dtype=dtype, device=DEV)
    pv, qv = wide_p[:, 1:, 5:5 + vocab], wide_q[:, :w - 1, 3:3 + vocab]
    pv.copy_(p)
    qv.copy_(q)
    tok = torch.empty((b, w), dtype=torch.int32, device=DEV)
    acc = torch.empty((b,), dtype=torch.int32, device=DEV)
    args = [t.to(DEV) for t in (draft, ua, us)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        N.dustin_verify_tokens(pv, qv, *args, tok, acc, n_draft=nd.to(DEV))
    side.synchronize()
    want = S.verify_tokens(H.f64(p), H.f64(q), draft.numpy(), nd.numpy(), H.f64(ua), H.f64(us))
    np.testing.assert_array_equal(tok.cpu().numpy(), want[0])
    np.testing.assert_array_equal(acc.cpu().numpy(), want[1])


def test_tokens_captured_graph_replays():
    p, q, draft, ua, us, nd = (t.to(DEV) for t in token_inputs(4, 3, 5000, torch.float32, 9))
    tok = torch.empty((4, 3), dtype=torch.int32, device=DEV)
    acc = torch.empty((4,), dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    N.dustin_verify_tokens(p, q, draft, ua, us, tok, acc)
    with torch.cuda.graph(g):
        N.dustin_verify_tokens(p, q, draft, ua, us, tok, acc)
    for seed in (10, 11):
        new = token_inputs(4, 3, 5000, torch.float32, seed)
        for t, x in zip((p, q, draft, ua, us), new):
            t.copy_(x)
        g.replay()
        H.sync()
        want = S.verify_tokens(H.f64(new[0]), H.f64(new[1]), new[2].numpy(), None, H.f64(new[3]),
                               H.f64(new[4]))
        np.testing.assert_array_equal(tok.cpu().numpy(), want[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [70, 5000, 40000])
def test_tokens_u_of_one_takes_the_last_token_with_mass(vocab, dtype):
    """However little mass the tail has: 1e-20 beside 1 changes no running sum
    of 53 bits, and is the last token all the same.  Tails in the same range as
    the rest, in another warp's, in another CTA's."""
    tails = [3, 40, vocab // 2 + 1, vocab - 1]
    p = torch.zeros((2 * len(tails), 2, vocab))
    for i, t in enumerate(tails):
        p[2 * i:2 * i + 2, :, 2] = 1.0
        p[2 * i:2 * i + 2, :, t] = 1e-20
    p = p.to(dtype)
    us = torch.tensor([1.0, float(np.nextafter(np.float32(1), np.float32(0)))]).repeat(len(tails))
    draft = torch.zeros((len(us), 1), dtype=torch.int32)
    tok, acc = check_tokens(p, None, draft, torch.ones((len(us), 1)), us, None)
    assert tok[0::2, 0].tolist() == tails and tok[1::2, 0].tolist() == [2] * len(tails)
    # The same out of a residual, and with u beyond 1.
    q = torch.zeros((len(us), 1, vocab))
    q[:, 0, 0] = 1.0
    tok, _ = check_tokens(p, q.to(dtype), draft, torch.ones((len(us), 1)), us * 2, None)
    assert tok[:, 0].tolist() == [t for t in tails for _ in range(2)]


def test_tokens_u_on_the_border_of_two_ranges():
    """t = u * total equal to the sum below a warp's range (8 entries here),
    where the range's start found as (sum to its end) - (its own sum) rounds to
    more than t.  Exactly: C_1 = 1 + 2^-52 = t, so token 8 is the first behind."""
    e = {0: 1.0, 1: 2.0 ** -52, 8: 1.0, 9: 2.0 ** -51, 16: 2.0, 24: 2.0 ** -52}
    p = torch.zeros((1, 1, 128))
    for j, x in e.items():
        p[0, 0, j] = x
    exact, total, below = {}, sum(Fraction(x) for x in e.values()), Fraction(0)
    for j, x in e.items():
        below += Fraction(x)
        exact[j] = below
    assert min(j for j in e if exact[j] > total / 4) == 8 and exact[1] == total / 4
    below, mine = 1 + 2.0 ** -52, 1 + 2.0 ** -51
    assert (below + mine) - mine > below             # in 53 bits
    none = torch.zeros((1, 0))
    tok, _ = run_tokens(p, None, none.int(), none, torch.tensor([0.25]), None)
    assert tok.tolist() == [[8]]


def test_tokens_sums_that_round_differently_one_by_one():
    """(1 + 2^-53) + 2^-53 is 1 = t in 53 bits, 1 + (2^-53 + 2^-53) is more: the
    warp that holds t has no entry behind it, and the draw stays with its
    entries, or those before, not with the ranges above."""
    e = {0: 1.0, 517: 2.0 ** -53, 645: 2.0 ** -53, 773: 1.0, 900: 1.0, 1024: 1.0}
    p = torch.zeros((200, 1, 8192))                  # 200 rows: one CTA each, 512 entries a warp
    for j, x in e.items():
        p[:, 0, j] = x
    total, below = sum(Fraction(x) for x in e.values()), Fraction(0)
    exact = [j for j in e if (below := below + Fraction(e[j])) > total * Fraction(0.2)]
    none = torch.zeros((200, 0))
    for u, want in ((0.2, exact[:1]), (0.25, (517, 645))):
        tok, _ = run_tokens(p, None, none.int(), none, torch.full((200,), u), None)
        assert set(tok[:, 0].tolist()) <= set(want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_entries_without_mass_at_the_draft(dtype):
    """Negative, NaN and infinite entries count as 0 in the acceptance too: such
    a target entry accepts no draft, such a draft entry every one with mass."""
    nan, inf, vocab = float("nan"), float("inf"), 40
    none = [0.0, -0.25, -0.75, nan, inf, -inf]
    pairs = [(x, y) for x in none + [0.5] for y in none + [0.5]]
    p = torch.zeros((len(pairs), 2, vocab))
    q = torch.zeros((len(pairs), 1, vocab))
    p[:, 0, 30], p[:, 1, 31] = 0.5, 1.0
    for i, (x, y) in enumerate(pairs):
        p[i, 0, 7], q[i, 0, 7] = x, y
    draft = torch.full((len(pairs), 1), 7, dtype=torch.int32)
    ua, us = torch.full((len(pairs), 1), 0.9), torch.zeros(len(pairs))
    tok, acc = check_tokens(p.to(dtype), q.to(dtype), draft, ua, us, None)
    assert acc.tolist() == [int(x == 0.5) for x, _ in pairs]
    assert tok[:, 0].tolist() == [7 if x == 0.5 else 30 for x, _ in pairs]
    tok, acc = check_tokens(p.to(dtype), None, draft, ua * 0.5, us, None)
    assert acc.tolist() == [int(x == 0.5) for x, _ in pairs]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [32768, 50001])
def test_tokens_edges_across_ctas(vocab, dtype):
    """Rows spread over eight CTAs: residuals without mass (summed again from
    the target's row), rows without mass, one-hot rows at the far end, u at 0,
    1 and NaN in each."""
    us = torch.tensor([0.0, 0.37, 0.9999, 1.0, float("nan")])
    n, g = len(us), I.generator(vocab)
    kinds = 6
    p = torch.softmax(3 * torch.randn((kinds * n, 2, vocab), generator=g), -1)
    q = p[:, :1].clone()
    ua = torch.ones((kinds * n, 1))
    draft = torch.randint(0, vocab, (kinds * n, 1), generator=g).int()
    at = [slice(i * n, (i + 1) * n) for i in range(kinds)]
    # kind 0: p equal to q, rejected: the residual is empty
    p[at[1]] = 0                                     # no mass at all
    p[at[2], 0] = 0
    p[at[2], 0, vocab - 1] = 0.25                    # one-hot, no mass in the first CTAs
    q[at[3]] = 1.0                                   # p below q everywhere but in one place
    q[at[3], 0, vocab - 5] = 0
    draft[at[3]] = 1
    p[at[4], 0, vocab // 16:] = 0                    # mass in the first CTA alone
    q[at[4]] = 0
    q[at[4], 0, vocab // 16:] = 1.0
    draft[at[4]] = vocab - 1
    q[at[5]] = 0                                     # accepted: the next row
    p, q = p.to(dtype), q.to(dtype)
    tok, acc = check_tokens(p, q, draft, ua, us.repeat(kinds), None)
    assert not acc[:5 * n].any() and acc[5 * n:].all()
    assert (tok[at[1], 0] == -1).all() and (tok[at[2], 0] == vocab - 1).all()
    assert (tok[at[3], 0] == vocab - 5).all() and (tok[at[4], 0] < vocab // 16).all()


# ----------------------------------------------------------------- compaction

def caches(b, hkv, n, d, page, layers, seed, spare=3):
    """layers of (K, V) logical [b][h][n][d], their storage and table."""
    g = I.generator(seed)
    logical = [[torch.randn((b, hkv, n, d), generator=g).to(torch.bfloat16) for _ in range(2)]
               for _ in range(layers)]
    if not page:
        return logical, [[x.to(DEV) for x in kv] for kv in logical], None
    pp = -(-n // page)
    table = torch.randperm(b * pp + spare, generator=g)[:b * pp].view(b, pp).int()
    stored = []
    for kv in logical:
        pools = []
        for x in kv:
            pool = torch.randn((b * pp + spare, hkv, page, d), generator=g).to(torch.bfloat16)
            padded = torch.cat([x, torch.zeros((b, hkv, pp * page - n, d), dtype=x.dtype)], 2)
            pool[table.long()] = padded.view(b, hkv, pp, page, d).transpose(1, 2)
            pools.append(pool.to(DEV))
        stored.append(pools)
    return logical, stored, table.to(DEV)


def read(x, table, n):
    if table is None:
        return x[:, :, :n]
    return x[table.long()].transpose(1, 2).flatten(2, 3)[:, :, :n]


COMPACT = [  # b, h_kv, d, n, k, layers, page of src, page of dst
    (1, 1, 64, 1, 1, 1, 0, 0),
    (2, 2, 128, 300, 45, 2, 0, 16),
    (3, 1, 64, 1000, 999, 1, 16, 0),
    (2, 8, 128, 2049, 130, 3, 48, 64),
    (1, 2, 128, 5000, 1500, 130, 16, 16),
]


@pytest.mark.parametrize("shape", COMPACT, ids=str)
@pytest.mark.parametrize("ragged", [False, True])
def test_compact_into_another_cache(shape, ragged):
    b, hkv, d, n, k, layers, p0, p1 = shape
    if layers > 100 and not ragged:
        n, k = 300, 40
    logical, stored, table = caches(b, hkv, n, d, p0, layers, seed=n + k)
    _, to, to_table = caches(b, hkv, k, d, p1, layers, seed=n + k + 1)
    g = I.generator(k)
    idx = torch.randint(0, n, (b, k), generator=g).int()          # any order, repeats
    k_len = torch.randint(0, k + 1, (b,), generator=g).int() if ragged else None
    before = [[x.clone() for x in kv] for kv in to]
    N.dustin_kv_compact([N.kv_desc(*kv, table) for kv in stored],
                        [N.kv_desc(*kv, to_table) for kv in to], hkv, d, n, idx.to(DEV),
                        k_len=None if k_len is None else k_len.to(DEV))
    H.sync()
    assert flags() == 0
    for l in range(layers):
        for x, y, y0 in zip(logical[l], to[l], before[l]):
            want = S.compact(x.float().numpy(), idx.numpy(), k_len,
                             read(y0, to_table, k).float().cpu().numpy().copy())
            np.testing.assert_array_equal(read(y, to_table, k).float().cpu().numpy(), want)


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("b,hkv,d,n,k", [(2, 2, 128, 700, 333), (1, 1, 64, 3000, 2900),
                                         (3, 2, 64, 150, 150), (2, 1, 128, 900, 129)])
def test_compact_in_place(b, hkv, d, n, k, page):
    logical, stored, table = caches(b, hkv, n, d, page, 2, seed=n + k)
    idx = I.random_sorted_indices(b, n, k, seed=n)
    idx[0, :k // 2] = torch.arange(k // 2)           # the front stays where it is
    idx[0, k // 2:] = torch.arange(n - (k - k // 2), n)
    k_len = torch.tensor([k] + [k - 7] * (b - 1)).int()
    descs = [N.kv_desc(*kv, table) for kv in stored]
    N.dustin_kv_compact(descs, descs, hkv, d, n, idx.to(DEV), k_len=k_len.to(DEV))
    H.sync()
    assert flags() == 0
    for kv, now in zip(logical, stored):
        for x, y in zip(kv, now):
            want = S.compact(x.float().numpy(), idx.numpy(), k_len, x.float().numpy().copy())
            np.testing.assert_array_equal(read(y, table, n).float().cpu().numpy(), want)


def test_compact_leaves_bad_entries_out():
    b, hkv, d, n, k, page = 2, 2, 64, 200, 20, 16
    logical, stored, table = caches(b, hkv, n, d, page, 1, seed=3)
    to = [[torch.zeros((b, hkv, k, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]]
    idx = I.random_sorted_indices(b, n, k, seed=4)
    idx[0, 3], idx[1, 5] = n, -1
    want = [S.compact(x.float().numpy(), idx.numpy(), None, np.zeros((b, hkv, k, d)))
            for x in logical[0]]
    N.dustin_kv_compact([N.kv_desc(*stored[0], table)], [N.kv_desc(*to[0])], hkv, d, n, idx.to(DEV))
    H.sync()
    assert flags() == INDEX_RANGE
    for x, y in zip(want, to[0]):
        np.testing.assert_array_equal(y.float().cpu().numpy(), x)
    table[1, 2] = 1 << 20
    N.dustin_kv_compact([N.kv_desc(*stored[0], table)], [N.kv_desc(*to[0])], hkv, d, n,
                        torch.arange(k, device=DEV).int().add(30).repeat(b, 1))
    H.sync()
    assert flags() == PAGE_RANGE
    descs = [N.kv_desc(*stored[0])]                  # the pools as contiguous caches
    N.dustin_kv_compact(descs, descs, hkv, d, page, torch.tensor([[3, 3], [1, 2]], device=DEV).int())
    H.sync()
    assert flags() == INDEX_ORDER


# --------------------------------------------------------------- shared pages

class Pages:
    """A page book on the GPU beside the oracle's, with one cache layer whose
    rows are filled with what their sequence and position should hold."""

    def __init__(self, lens, per, page, pages, hkv=2, d=64, layers=2, seed=0):
        g = I.generator(seed)
        self.per, self.page, self.hkv, self.d = per, page, hkv, d
        perm = iter(torch.randperm(pages, generator=g).tolist())
        table = [[next(perm) if x * page < n else -1 for x in range(per)] for n in lens]
        count = [0] * pages
        for row in table:
            for x in row:
                if x >= 0:
                    count[x] += 1
        self.book = S.PageBook(table, lens, count, page)
        self.table, self.lens, self.count = (torch.tensor(x, dtype=torch.int32, device=DEV)
                                             for x in (table, lens, count))
        self.pools = [[torch.randn((pages, hkv, page, d), generator=g).to(torch.bfloat16).to(DEV)
                       for _ in range(2)] for _ in range(layers)]

    def same(self):
        H.sync()
        assert self.table.tolist() == self.book.table
        assert self.lens.tolist() == self.book.seq_len
        assert self.count.tolist() == self.book.refcount

    def fork(self, parents, children):
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        N.dustin_kv_fork(self.table, self.lens, self.count, self.page, t(parents), t(children))
        skipped = self.book.fork(parents, children)
        self.same()
        assert flags() == (INDEX_RANGE if skipped else 0)
        return skipped

    def resize(self, seqs, new, extra=0):
        t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)
        copies = torch.full((len(seqs), 2), -7, dtype=torch.int32, device=DEV)
        before = [[x.clone() for x in kv] for kv in self.pools]
        kvs = [N.kv_desc(*kv, self.table) for kv in self.pools]
        N.dustin_kv_resize(self.table, self.lens, self.count, self.page, t(seqs), t(new), copies,
                           kvs=kvs, h_kv=self.hkv, d=self.d)
        want, starved = self.book.resize(seqs, [0] * len(seqs) if new is None else new)
        self.same()
        assert copies.tolist() == want
        assert flags() == (NO_PAGES if starved else 0) | extra
        for kv, now in zip(before, self.pools):
            for x, y in zip(kv, now):
                for src, dst in want:
                    if src >= 0:
                        x[dst] = x[src]
                assert torch.equal(x, y)
        return want, starved


@pytest.mark.parametrize("page", [16, 48])
def test_pages_turn_of_a_serving_loop(page):
    p = Pages([37, 3 * page, 0, 0, 0, 0, 0], 8, page, 40, seed=page)
    p.fork([0, 1, 0, 0], [2, 3, 4, 5])
    copies, _ = p.resize([2, 3, 4, 0], [41, 3 * page + 5, 37 + 2 * page, 38])
    assert [c[0] >= 0 for c in copies] == [True, False, True, True]
    p.resize([2, 4, 3], [39, 0, page])                           # back to the accepted tokens
    p.resize([5, 6, 0], [38, 1, 8 * page])                       # the last sharer keeps its page
    p.fork([6], [4])
    p.resize([0, 1, 2, 3, 4, 5, 6], None)
    assert p.count.tolist() == [0] * 40


def test_pages_grow_until_none_is_left():
    p = Pages([20, 0, 0, 0], 6, 16, 8, seed=4)
    p.fork([0], [1])
    assert p.resize([1, 2, 3, 0], [21, 80, 30, 10])[1] == [2]    # six free, 5 + 2 wanted
    assert p.resize([3, 2], [16, 96])[1] == [1]
    assert p.resize([2, 0, 3], [0, 11, 80])[1] == []


def test_pages_left_out_entries():
    p = Pages([20, 33, 0, 5], 4, 16, 20, seed=5)
    assert p.fork([0, 0, 1, 9, 2, 0], [2, 2, 1, 2, 3, 3]) == [1, 2, 3, 4, 5]
    p2 = Pages([20, 33, 0, 0], 4, 16, 20, seed=6)
    assert p2.fork([2, 0], [3, 2]) == [0]                        # a parent that is a child
    p2.resize([1, 1, -1, 4, 3], [5, 9, 9, 9, 65], extra=INDEX_RANGE)


@pytest.mark.parametrize("children,pages,n", [(100, 4096, 1000), (512, 70000, 333), (1000, 2500, 17)])
def test_pages_many_sequences(children, pages, n):
    per = -(-(n + 40) // 16)
    p = Pages([n, n - 9] + [0] * children, per, 16, pages, hkv=1, layers=1, seed=children)
    kids = [int(x) + 2 for x in torch.randperm(children, generator=I.generator(1))]
    p.fork([x % 2 for x in kids], kids)
    g = I.generator(2)
    p.resize(kids, [n + int(x) for x in torch.randint(-16, 40, (children,), generator=g)])
    p.resize(kids[::2], [int(x) for x in torch.randint(0, n + 40, (len(kids[::2]),), generator=g)])
    assert p.book.consistent()
    p.resize(kids, None)


def test_pages_without_caches_and_with_bad_page_ids():
    p = Pages([20, 0], 4, 16, 8, seed=8)
    p.table[0, 1] = 99                               # a page outside the pool: skipped, flagged
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    copies = t([[0, 0]])
    N.dustin_kv_resize(p.table, p.lens, p.count, 16, t([0]), t([3]), copies)
    H.sync()
    assert flags() == PAGE_RANGE and p.lens.tolist() == [3, 0] and copies.tolist() == [[-1, -1]]
