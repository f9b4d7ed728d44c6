"""Log probabilities, entropies and alternatives on the GPU against the oracle.

Tolerances.  With d = x - max exact to 2^-24 of itself, a weight e^(scale d) is off by
scale |d| 2^-23 + 2^-22 (the exponential) of itself, and weights count only where
scale |d| < 60 or so; the sum of n weights in fp32, 152 thousand in at most 512 lanes
and a tree, by another 2^-24 * 400.  ln l is so off by 4e-5 at the very most (weights
of scale |d| = 60 are e^-60 of the sum: those that matter, below 20, give 2e-6 +
2.4e-5); a log probability z by that and 2^-22 |z|; the entropy, whose terms are
weights times scale |d|, by 4e-5 (1 + entropy).  Ids are exact."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as Q
from sparse_kv_verification_gb300 import build, inputs as I, native as N
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
INDEX_RANGE = 1
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return N.load()


def flags():
    f = ctypes.c_uint32(0)
    N.load().dustin_device_status(ctypes.byref(f))
    return f.value


def run(x, tokens, top, scale=1.0, n_rows=None):
    b, w, _ = x.shape
    full = lambda *s: torch.full(s, -7.0, device=DEV)
    lp, ent, lse = full(b, w, tokens.shape[-1]), full(b, w), full(b, w)
    ids, best = torch.full((b, w, top), -7, dtype=torch.int32, device=DEV), full(b, w, top)
    N.dustin_token_logprobs(x, tokens.to(DEV), lp, ent, lse, ids, best, scale=scale,
                            n_rows=None if n_rows is None else torch.tensor(n_rows, dtype=torch.int32,
                                                                            device=DEV))
    H.sync()
    return [t.double().cpu().numpy() for t in (lp, ent, lse)] + [ids.cpu().numpy(),
                                                                 best.double().cpu().numpy()]


def close(got, want, tol):
    got, want = np.asarray(got), np.asarray(want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.all(np.abs(got[fin] - want[fin]) <= np.broadcast_to(tol, want.shape)[fin])


def check(x, tokens, top, scale=1.0, n_rows=None):
    lp, ent, lse, ids, best = got = run(x.to(DEV) if not x.is_cuda else x, tokens, top, scale, n_rows)
    f = x.double().cpu().numpy()
    s = float(np.float32(scale))
    for i in range(x.shape[0]):
        for t in range(x.shape[1]):
            if n_rows is not None and t >= n_rows[i]:
                assert all((a[i, t] == -7).all() for a in got)           # left as they were
                continue
            r_lp, r_ent, r_lse, r_ids, r_best = Q.logprobs(f[i, t], s, tokens[i, t].tolist(), top)
            np.testing.assert_array_equal(ids[i, t], r_ids)
            close(lp[i, t], r_lp, 4e-5 + 2.0 ** -22 * np.abs(r_lp))
            close(best[i, t], r_best, 4e-5 + 2.0 ** -22 * np.abs(r_best))
            close(lse[i, t], r_lse, 4e-5 + 2.0 ** -22 * abs(r_lse))
            close(ent[i, t], r_ent, 4e-5 * (1 + abs(r_ent)))
    return got


def inputs(b, w, vocab, dtype, m, seed, sharp=2.5):
    g = I.generator(seed)
    x = (sharp * torch.randn((b, w, vocab), generator=g)).to(dtype)
    return x, torch.randint(0, vocab, (b, w, m), generator=g).int()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,w,vocab,m,top", [(1, 1, 1, 1, 1), (1, 2, 7, 3, 5), (3, 4, 129, 2, 20),
                                             (1, 1, 4099, 0, 64), (2, 3, 32000, 1, 5),
                                             (5, 2, 50257, 2, 20), (400, 1, 1000, 1, 3),
                                             (1, 2, 152064, 1, 64), (40, 4, 2049, 512, 0),
                                             (2, 1, 65536, 0, 0), (100, 2, 257, 1, 17)])
def test_parity(b, w, vocab, m, top, dtype):
    x, tokens = inputs(b, w, vocab, dtype, m, seed=vocab + b)
    check(x, tokens, top)
    assert flags() == 0


@pytest.mark.parametrize("scale", [1e-3, 0.7, 30.0])
def test_temperatures_and_ragged_windows(scale):
    x, tokens = inputs(4, 5, 3001, torch.float32, 2, seed=3)
    check(x, tokens, 7, scale, n_rows=[5, 0, 3, 9])
    check(x + 500.0, tokens, 7, scale, n_rows=[-1, 5, 1, 2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_at_any_element_and_stride(dtype):
    """Odd starts, rows cut out of longer ones whose other entries would win, shared
    rows."""
    x, tokens = inputs(3, 2, 1234, dtype, 1, seed=1)
    for pad in (1, 2, 3, 5, 8, 13):
        wide = torch.full((3, 2, 1234 + 2 * pad + 1), 1e4, dtype=dtype, device=DEV)
        wide[..., pad:pad + 1234] = x.to(DEV)
        check(wide[..., pad:pad + 1234], tokens, 12)
    check(x[:1, :1].to(DEV).expand(3, 2, 1234), tokens, 12)
    check(x.to(DEV).transpose(0, 1), tokens.transpose(0, 1).contiguous(), 12)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [100, 5000, 152064])
def test_ties_go_to_the_lowest_id(dtype, vocab):
    """Flat rows, few values, -0 and +0, rising and falling rows."""
    j = torch.arange(vocab)
    rows = [torch.zeros(vocab), torch.where(j % 2 == 0, 0.0, -0.0), (j % 3).float(), (j // 7 % 5).float(),
            j.float() / 4096, -j.float() / 4096, torch.full((vocab,), -3.5), (j >= vocab - 3).float()]
    x = torch.stack(rows).to(dtype).view(len(rows), 1, vocab)
    check(x, torch.zeros((len(rows), 1, 1), dtype=torch.int32), 64)
    check(x, torch.zeros((len(rows), 1, 1), dtype=torch.int32), 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [70, 40000])
def test_banned_tokens_nan_and_infinities(dtype, vocab):
    x, tokens = inputs(9, 1, vocab, dtype, 2, seed=9)
    x[0] = -INF                                        # nothing allowed
    x[1] = -INF
    x[1, 0, vocab - 3] = 2.0                           # one token allowed
    x[2, 0, ::2] = -INF
    x[3, 0, vocab // 2] = NAN
    x[4, 0, 5] = INF
    x[5] = NAN
    x[6] = -INF
    x[6, 0, vocab - 1] = NAN
    x[7, 0, :] = -INF
    x[7, 0, 10:40] = 1.5
    x[8, 0, 3], x[8, 0, 4] = 3e38 if dtype == torch.float32 else 1e38, -3e38
    tokens[1, 0, 0] = vocab - 3
    tokens[7, 0, 0] = 12
    check(x, tokens, 64)
    check(x, tokens, 1)
    assert flags() == 0


def test_tokens_outside_the_vocabulary():
    x, tokens = inputs(1, 3, 50, torch.float32, 3, seed=4)
    tokens[0, 0] = torch.tensor([-1, 3, -1])           # no token: no flag
    check(x, tokens, 2)
    assert flags() == 0
    tokens[0, 1] = torch.tensor([50, -2, 2 ** 31 - 1])
    lp = check(x, tokens, 2)[0]
    assert np.isneginf(lp[0, 1]).all() and flags() == INDEX_RANGE


def test_optional_outputs_streams_and_graphs():
    x, tokens = inputs(3, 4, 20000, torch.bfloat16, 1, seed=8)
    want = run(x.to(DEV), tokens, 6)
    x, tokens = x.to(DEV), tokens.to(DEV)
    lse = torch.zeros((3, 4), device=DEV)
    N.dustin_token_logprobs(x, None, None, lse=lse)    # one thing alone
    np.testing.assert_array_equal(lse.double().cpu().numpy(), want[2])
    lp = torch.zeros((3, 4, 1), device=DEV)
    ids, best = torch.zeros((3, 4, 6), dtype=torch.int32, device=DEV), torch.zeros((3, 4, 6), device=DEV)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    H.sync()
    with torch.cuda.graph(graph, stream=stream):
        N.dustin_token_logprobs(x, tokens, lp, top_ids=ids, top_logprobs=best)
    for _ in range(2):
        lp.zero_(), ids.zero_(), best.zero_()
        graph.replay()
        H.sync()
        for got, ref in zip((lp, ids, best), (want[0], want[3], want[4])):
            np.testing.assert_array_equal(got.double().cpu().numpy(), ref)


def test_equal_calls_give_equal_bits_and_peaks_are_exact():
    x, tokens = inputs(2, 2, 152064, torch.float32, 1, seed=5)
    a, b = run(x.to(DEV), tokens, 20), run(x.to(DEV), tokens, 20)
    for p, q in zip(a, b):
        np.testing.assert_array_equal(p, q)
    x[0, 0, 77] = 200.0                                # certain: logprob 0, entropy 0
    tokens[0, 0, 0] = 77
    lp, ent, lse, ids, _ = check(x, tokens, 3)
    assert lp[0, 0, 0] == 0 and ent[0, 0] == 0 and ids[0, 0, 0] == 77


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_small_weights_behind_large_ones(dtype):
    """2^26 logits of which each thread of eight CTAs meets one of 0 first and 2^14 of
    -17.5 after it: each of these is less than half a step of the sum so far, together
    they are 4e-4 of it."""
    vocab, v = 1 << 26, 4 if dtype == torch.float32 else 8
    j = torch.arange(vocab, device=DEV)
    first = (j % (vocab // 8) < 512 * v) & (j % v == 0)
    n = int(first.sum())
    x = torch.where(first, 0.0, -17.5).to(dtype).view(1, 1, vocab)
    tokens = torch.tensor([[[0, 1, vocab - 1]]], dtype=torch.int32)
    lp, ent, lse, ids, best = run(x, tokens, 2)
    small = math.exp(-17.5)
    total = n + (vocab - n) * small
    r_lse, r_ent = math.log(total), math.log(total) + (vocab - n) * small * 17.5 / total
    assert n == 4096 and abs(math.log(n) - r_lse) > 4e-4
    close(lse, [[r_lse]], 4e-5)
    close(lp, [[[-r_lse, -17.5 - r_lse, -17.5 - r_lse]]], 4e-5 + 2.0 ** -22 * 30)
    close(ent, [[r_ent]], 4e-5 * (1 + r_ent))
    np.testing.assert_array_equal(ids, [[[0, v]]])
