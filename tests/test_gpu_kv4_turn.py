"""The 4-bit cache, the attention over it and the log probabilities together with the
selection and the verification of tokens, as a serving loop uses them: prompts are
written to paged caches, then turns of selection, attention of the window's rows over
the selected positions and the bf16 window, log probabilities and verification of the
drafts, and the accepted rows written behind the cache.  Every step is held to the
oracle, fed with what the step before produced; then the same turns as one captured
graph, replayed, have to leave the same bits.

Tolerances: those of the attention's and the log probabilities' tests; the rest is
exact."""
import numpy as np
import pytest
import torch

from oracle import dustin_oracle as O
from oracle import kv4_oracle as Q
from oracle import serving_oracle as S
from sparse_kv_verification_gb300 import build, inputs as I, native as N
from tests import gpu_harness as H
from tests.test_gpu_kv4 import check, f64, flags
from tests.test_gpu_logprobs import close

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, HKV, HQ, W, VOCAB, TOP, CAP, K, PAGE = 3, 2, 6, 4, 301, 5, 320, 96, 16
SCALE = 0.8


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return N.load()


class Server:
    def __init__(self, d):
        g = I.generator(d)
        z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=DEV)
        self.d, rec = d, N.kv4_record_size(d)
        per = CAP // PAGE
        self.table = torch.randperm(B * per, generator=g).int().view(B, per).to(DEV)
        self.pool = torch.full((B * per, HKV, PAGE, rec), 0xff, dtype=torch.uint8, device=DEV)
        self.lens = torch.tensor([200, 129, 256], dtype=torch.int32, device=DEV)
        self.prompt = [torch.randn((B, HKV, 256, d), generator=g).bfloat16().to(DEV) for _ in range(2)]
        self.q, self.o = z(B, HQ, W, d), z(B, HQ, W, d)
        self.win = [z(B, HKV, W, d), z(B, HKV, W, d)]
        self.lse = z(B, HQ, W, t=torch.float32)
        self.score = z(B, CAP, t=torch.float32)
        self.idx = z(B, K, t=torch.int32)
        self.head = torch.randn((HQ * d, VOCAB), generator=g).to(DEV) / 8
        self.draft = z(B, W - 1, t=torch.int32)
        self.given = z(B, W, 1, t=torch.int32)
        self.ua, self.us = z(B, W - 1, t=torch.float32), z(B, t=torch.float32)
        self.lp, self.ent = z(B, W, 1, t=torch.float32), z(B, W, t=torch.float32)
        self.ids, self.best = z(B, W, TOP, t=torch.int32), z(B, W, TOP, t=torch.float32)
        self.tokens, self.acc = z(B, W, t=torch.int32), z(B, t=torch.int32)
        self.ws = N.workspace(N.dustin_kv4_verify_attn_workspace_size(B, HQ, HKV, d, W, K), DEV)
        N.dustin_kv4_write([N.kv_desc(*self.prompt)], [self.kv4()], B, HKV, d, CAP, 256, w_len=self.lens)

    def kv4(self):
        return N.kv4_desc(self.pool, self.table, 1, -2)

    def load(self, turn):
        g = I.generator(100 + turn)
        r = lambda *s: torch.randn(s, generator=g)
        self.q.copy_(r(*self.q.shape))
        for x in self.win:
            x.copy_(r(*x.shape))
        self.score.copy_(torch.rand(self.score.shape, generator=g))
        self.draft.copy_(torch.randint(0, VOCAB, self.draft.shape, generator=g))
        self.ua.copy_(torch.rand(self.ua.shape, generator=g) * 0.01)
        self.us.copy_(torch.rand(self.us.shape, generator=g))

    def turn(self):
        # Scores behind a sequence's end lose; sequences shorter than the budget
        # take their own length of it.
        at = torch.arange(CAP, device=DEV)
        self.masked = torch.where(at[None] < self.lens[:, None], self.score, -1.0)
        N.dustin_hybrid_topk(self.masked, None, K, 0, 0, 1.0, -1, N.DUSTIN_NORM_NONE, self.idx)
        N.dustin_kv4_verify_attn(self.q, self.kv4(), HKV, CAP, K, self.d ** -0.5, self.o, self.lse,
                                 self.ws, idx=self.idx, win=N.kv_desc(*self.win))
        hidden = self.o.transpose(1, 2).reshape(B, W, HQ * self.d).float()
        self.logits = (hidden.unsqueeze(-1) * self.head).sum(-2)
        self.given[:, :W - 1, 0].copy_(self.draft)
        self.given[:, W - 1].fill_(-1)                   # no draft for the last row
        N.dustin_token_logprobs(self.logits, self.given, self.lp, self.ent, None, self.ids, self.best,
                                scale=SCALE)
        self.p = torch.softmax(self.logits * SCALE, -1)
        N.dustin_verify_tokens(self.p, None, self.draft, self.ua, self.us, self.tokens, self.acc)
        N.dustin_kv4_write([N.kv_desc(*self.win)], [self.kv4()], B, HKV, self.d, CAP, W,
                           start=self.lens, w_len=self.acc + 1)
        self.lens += self.acc + 1

    def state(self):
        H.sync()
        return [x.clone() for x in (self.pool, self.lens, self.o, self.lse, self.idx, self.lp, self.ent,
                                    self.ids, self.best, self.tokens, self.acc)]

    def records(self):
        """What the cache holds, [b][h_kv][CAP][record]."""
        x = self.pool[self.table.long()].transpose(1, 2)
        return x.reshape(B, HKV, CAP, -1).cpu().numpy()


def check_turn(s):
    rec, lens = s.records(), s.lens.tolist()
    s.turn()
    H.sync()
    want_idx = O.hybrid_select(f64(s.masked), None, K, 0, 0, 1.0, -1, O.NORM_NONE)
    np.testing.assert_array_equal(s.idx.cpu().numpy(), want_idx)
    k, v = Q.dequantise(rec, s.d, 1, -2)
    win = [f64(x) for x in s.win]
    check(s.o, s.lse, Q.attention(f64(s.q), k, v, s.d ** -0.5, list(want_idx), *win), large=2.0)
    logits, given = f64(s.logits), s.given.cpu().numpy()
    for i in range(B):
        for t in range(W):
            lp, ent, _, ids, best = Q.logprobs(logits[i, t], float(np.float32(SCALE)), given[i, t], TOP)
            np.testing.assert_array_equal(s.ids[i, t].cpu().numpy(), ids)
            close(f64(s.lp[i, t]), lp, 4e-5 + 2.0 ** -22 * np.abs(lp))
            close(f64(s.best[i, t]), best, 4e-5 + 2.0 ** -22 * np.abs(best))
            close(f64(s.ent[i, t]), ent, 4e-5 * (1 + ent))
    tokens, acc = S.verify_tokens(f64(s.p), None, s.draft.cpu().numpy(), None, f64(s.ua), f64(s.us))
    np.testing.assert_array_equal(s.tokens.cpu().numpy(), tokens)
    np.testing.assert_array_equal(s.acc.cpu().numpy(), acc)
    for i in range(B):
        m = int(acc[i]) + 1
        rec[i, :, lens[i]:lens[i] + m] = Q.quantise(*(x[i, :, :m] for x in win), 1, -2)
    np.testing.assert_array_equal(s.records(), rec)
    assert s.lens.tolist() == [n + int(a) + 1 for n, a in zip(lens, acc)] and flags() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_turns_against_the_oracle_and_captured(d):
    flags()
    s, graphed = Server(d), Server(d)
    rec = s.records()
    for i, n in enumerate(s.lens.tolist()):
        np.testing.assert_array_equal(rec[i, :, :n], Q.quantise(*(f64(x[i, :, :n]) for x in s.prompt), 1, -2))
        assert (rec[i, :, n:] == 0xff).all()
    kept = [graphed.pool.clone(), graphed.lens.clone()]
    stream = torch.cuda.Stream()
    graphed.load(0)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graphed.turn()                                   # everything allocated and loaded once
        graphed.pool.copy_(kept[0]), graphed.lens.copy_(kept[1])
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
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
