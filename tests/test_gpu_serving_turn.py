"""The serving operators together, as a server would use them: samples forked
from prompts on shared pages, then turns of grow (copy on write), attention
over the shared prefix, the own pages and the window, verification of the
drafted tokens and shrinking to the accepted ones; at the end each sample's
cache is compacted in place.  Every step is held to the oracle, fed with what
the step before produced; then the same turns as one captured graph, replayed,
have to leave the same bits.

Tolerances: those of the attention test (bf16 weights and results, 2^-8 of
sum_j p_j |v_j| + |o|, plus 2^-13); everything else is exact."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from sparse_kv_verification_gb300 import build, inputs as I, native as N
from tests import gpu_harness as H
from tests.test_gpu_serving import flags

pytestmark = pytest.mark.gpu
DEV = "cuda"
PER, HKV, HQ, D, W, VOCAB, PAGES, ROW_PAGES = 3, 2, 6, 64, 4, 97, 64, 8


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return N.load()


class Server:
    """Two prompts (sequences 0 and 1) and PER samples of each."""

    def __init__(self, page, prompts):
        g = I.generator(page)
        self.page, self.shared = page, min(prompts) // page
        self.b = 2 * PER
        n_seqs = 2 + self.b
        table = torch.full((n_seqs, ROW_PAGES), -1, dtype=torch.int32)
        perm = torch.randperm(PAGES, generator=g).int()
        count = torch.zeros(PAGES, dtype=torch.int32)
        at = 0
        for i, n in enumerate(prompts):
            m = -(-n // page)
            table[i, :m] = perm[at:at + m]
            count[perm[at:at + m].long()] = 1
            at += m
        lens = list(prompts) + [0] * self.b
        self.book = S.PageBook(table.tolist(), lens, count.tolist(), page)
        self.table, self.count = table.to(DEV), count.to(DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.pool = [torch.randn((PAGES, HKV, page, D), generator=g).to(torch.bfloat16).to(DEV)
                     for _ in range(2)]
        self.head = torch.randn((HQ * D, VOCAB), generator=g).to(DEV) / 8
        self.seqs = torch.arange(2, n_seqs, dtype=torch.int32, device=DEV)
        self.copies = torch.empty((self.b, 2), dtype=torch.int32, device=DEV)
        self.copies_back = torch.empty_like(self.copies)
        z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=DEV)
        self.q, self.o = z(self.b, HQ, W, D), z(self.b, HQ, W, D)
        self.win = [z(self.b, HKV, W, D), z(self.b, HKV, W, D)]
        self.lse = z(self.b, HQ, W, t=torch.float32)
        self.p_draft = z(self.b, W - 1, VOCAB, t=torch.float32)
        self.draft = z(self.b, W - 1, t=torch.int32)
        self.ua, self.us = z(self.b, W - 1, t=torch.float32), z(self.b, t=torch.float32)
        self.tokens, self.acc = z(self.b, W, t=torch.int32), z(self.b, t=torch.int32)
        self.n_prefix = self.shared * page
        self.n_own = (ROW_PAGES - self.shared) * page
        self.ws = N.workspace(N.dustin_prefix_verify_attn_workspace_size(
            self.b, 2, HQ, HKV, D, W, self.n_prefix, self.n_own), DEV)

    def fork(self):
        parent = torch.arange(2, dtype=torch.int32, device=DEV).repeat_interleave(PER)
        N.dustin_kv_fork(self.table, self.lens, self.count, self.page, parent, self.seqs)

    def load(self, turn):
        """The turn's inputs: what a model and its draft would produce."""
        g = I.generator(100 + turn)
        r = lambda *s: torch.randn(s, generator=g)
        self.q.copy_(r(*self.q.shape))
        for x in self.win:
            x.copy_(r(*x.shape))
        draft_p = torch.softmax(r(*self.p_draft.shape), -1)
        self.p_draft.copy_(draft_p)
        self.draft.copy_(torch.multinomial(draft_p.view(-1, VOCAB), 1, generator=g).view(self.b, W - 1))
        self.ua.copy_(torch.rand(self.ua.shape, generator=g))
        self.us.copy_(torch.rand(self.us.shape, generator=g))

    def kv(self, rows=slice(None), first=0):
        return N.kv_desc(*self.pool, self.table[rows, first:])

    def resize(self, new_len, copies):
        N.dustin_kv_resize(self.table, self.lens, self.count, self.page, self.seqs, new_len, copies,
                           kvs=[self.kv()], h_kv=HKV, d=D)

    def turn(self):
        old = self.lens[2:].clone()
        own = old - self.n_prefix
        self.resize(old + W, self.copies)
        # The window's rows into their pages.
        at = old.long().view(-1, 1) + torch.arange(W, device=DEV)
        pages = self.table[2:].gather(1, at // self.page).long()
        for pool, x in zip(self.pool, self.win):
            pool[pages, :, at % self.page] = x.transpose(1, 2)
        N.dustin_prefix_verify_attn(
            self.q, self.kv(slice(0, 2)), self.kv(slice(2, None), self.shared), HKV, 2,
            self.n_prefix, self.n_own, D ** -0.5, self.o, self.lse, self.ws,
            win=N.kv_desc(*self.win), own_len=own)
        hidden = self.o.transpose(1, 2).reshape(self.b, W, HQ * D).float()
        self.p = torch.softmax((hidden.unsqueeze(-1) * self.head).sum(-2), -1)
        N.dustin_verify_tokens(self.p, self.p_draft, self.draft, self.ua, self.us, self.tokens,
                               self.acc)
        # The last token drawn has no K/V yet.
        self.resize(old + 1 + self.acc, self.copies_back)

    def state(self):
        H.sync()
        return [x.clone() for x in (self.table, self.lens, self.count, *self.pool, self.o, self.lse,
                                    self.tokens, self.acc)]

    def rows(self, seq, x):
        """A sequence's rows of pool x as the book has it: [h_kv][n][d]."""
        n = self.book.seq_len[seq]
        pages = self.book.table[seq][:self.book.pages(n)]
        return self.pool[x][pages].transpose(0, 1).reshape(HKV, -1, D)[:, :n]


def check_turn(s):
    """One turn beside the oracle's.  `kept` are the sequences' rows as plain
    tensors, before the turn."""
    kept = [[s.rows(i, x).clone() for i in range(2 + s.b)] for x in range(2)]
    old = list(s.book.seq_len[2:])
    s.turn()
    H.sync()
    seqs = list(range(2, 2 + s.b))
    want_copies, starved = s.book.resize(seqs, [n + W for n in old])
    assert not starved and s.copies.tolist() == want_copies

    f = lambda x: x.double().cpu().numpy()
    prefix = [np.stack([f(kept[x][g][:, :s.n_prefix]) for g in range(2)]) for x in range(2)]
    own = []
    for x in range(2):
        a = np.zeros((s.b, HKV, s.n_own, D))
        for i, n in enumerate(old):
            a[i, :, :n - s.n_prefix] = f(kept[x][2 + i][:, s.n_prefix:])
        own.append(a)
    win = [f(x) for x in s.win]
    at = lambda v: S.prefix_attention(f(s.q), prefix[0], v(prefix[1]), own[0], v(own[1]), 2,
                                      D ** -0.5, None, [n - s.n_prefix for n in old], win[0],
                                      v(win[1]))
    (o, lse), spread = at(lambda v: v), at(np.abs)[0]
    assert np.all(np.abs(f(s.o) - o) <= 2.0 ** -8 * (spread + np.abs(o)) + 2.0 ** -13)
    np.testing.assert_allclose(f(s.lse), lse, atol=2e-4, rtol=0)

    tokens, acc = S.verify_tokens(f(s.p), f(s.p_draft), s.draft.cpu().numpy(), None, f(s.ua),
                                  f(s.us))
    np.testing.assert_array_equal(s.tokens.cpu().numpy(), tokens)
    np.testing.assert_array_equal(s.acc.cpu().numpy(), acc)

    s.book.resize(seqs, [n + 1 + int(a) for n, a in zip(old, acc)])
    assert s.table.tolist() == s.book.table and s.lens.tolist() == s.book.seq_len
    assert s.count.tolist() == s.book.refcount and s.book.consistent()
    assert flags() == 0
    # Rows: the prompts' untouched, the samples' followed by the accepted ones.
    for x in range(2):
        for i in range(2 + s.b):
            want = kept[x][i]
            if i >= 2:
                want = torch.cat([want, s.win[x][i - 2, :, :1 + int(acc[i - 2])]], 1)
            assert torch.equal(s.rows(i, x), want)


@pytest.mark.parametrize("page,prompts", [(16, (40, 37)), (32, (64, 70))])
def test_turns_against_the_oracle_and_captured(page, prompts):
    flags()
    s, graphed = Server(page, prompts), Server(page, prompts)
    for x in (s, graphed):
        x.fork()
    s.book.fork([0] * PER + [1] * PER, list(range(2, 2 + s.b)))
    assert s.table.tolist() == s.book.table and s.count.tolist() == s.book.refcount
    start = [x.clone() for x in (graphed.table, graphed.lens, graphed.count, *graphed.pool)]
    back = lambda: [x.copy_(y) for x, y in zip((graphed.table, graphed.lens, graphed.count,
                                                *graphed.pool), start)]
    graphed.load(0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graphed.turn()                 # everything allocated and loaded once
        back()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            graphed.turn()
        for turn in range(3):
            graphed.load(turn)
            graph.replay()
    torch.cuda.current_stream().wait_stream(stream)
    for turn in range(3):
        s.load(turn)
        check_turn(s)
    for x, y in zip(s.state(), graphed.state()):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))

    # The caches cut down in place to the shared pages and a choice behind them.
    g = I.generator(7)
    lens = s.book.seq_len[2:]
    most = max(lens)
    idx = torch.zeros((s.b, most), dtype=torch.int32)
    k_len = []
    for i, n in enumerate(lens):
        chosen = torch.randperm(n - s.n_prefix, generator=g)[:1 + (n - s.n_prefix) // 2]
        row = torch.cat([torch.arange(s.n_prefix), s.n_prefix + chosen.sort().values]).int()
        idx[i, :len(row)] = row
        k_len.append(len(row))
    before = [[s.rows(i, x).clone() for i in range(2 + s.b)] for x in range(2)]
    own = [s.kv(slice(2, None))]
    N.dustin_kv_compact(own, own, HKV, D, most, idx.to(DEV),
                        k_len=torch.tensor(k_len, dtype=torch.int32, device=DEV))
    s.resize(torch.tensor(k_len, dtype=torch.int32, device=DEV), s.copies)
    s.book.resize(list(range(2, 2 + s.b)), k_len)
    H.sync()
    assert s.table.tolist() == s.book.table and s.count.tolist() == s.book.refcount
    assert flags() == 0
    for x in range(2):
        for i in range(2 + s.b):
            want = before[x][i]
            if i >= 2:
                want = want[:, idx[i - 2, :k_len[i - 2]].long().to(DEV)]
            assert torch.equal(s.rows(i, x), want)
    s.resize(None, s.copies)
    s.book.resize(list(range(2, 2 + s.b)), [0] * s.b)
    H.sync()
    assert s.count.tolist() == s.book.refcount and s.book.consistent()
