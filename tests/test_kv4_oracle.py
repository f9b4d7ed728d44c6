"""Pins of the 4-bit cache's and the log probabilities' oracle: the formats'
tables, brute force over every code and scale, closed forms."""
import numpy as np
import pytest

from oracle import dustin_oracle as O
from oracle import kv4_oracle as Q


def test_the_formats():
    assert Q.record_size(64) == 80 and Q.record_size(128) == 144
    assert Q.e4m3([0, 1, 7, 8, 0x38, 0x7e]).tolist() == [0, 2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1, 448]
    assert np.isnan(Q.e4m3([0x7f, 0xff])).all() and Q.e4m3([0x80, 0xb8]).tolist() == [0, -1]
    assert np.all(np.diff(Q.SCALES) > 0)


def test_quantising_takes_the_nearest_scale_and_codes():
    """Against an exhaustive search; ties go to the even one."""
    r = np.random.default_rng(0)
    x = np.ldexp(r.integers(-255, 256, (400, 16)), r.integers(-12, 4, (400, 1))).astype(np.float64)
    codes, scale = Q.quantise_blocks(x, 0)
    for row, c, s in zip(x, codes, scale):
        off = np.abs(6 * Q.SCALES - min(np.abs(row).max(), 6 * 448))
        best = np.nonzero(off == off.min())[0]
        assert s == (best[0] if len(best) == 1 else best[best % 2 == 0][0])
        for y, code in zip(row, c):
            if s == 0:
                assert code % 8 == 0
                continue
            off = np.abs(Q.STEPS * Q.SCALES[s] - abs(y))
            best = np.nonzero(off == off.min())[0]
            assert code % 8 == (best[0] if len(best) == 1 else best[best % 2 == 0][0])
            assert code // 8 == (1 if np.signbit(y) else 0)


@pytest.mark.parametrize("d,k_exp,v_exp", [(64, 0, 0), (128, -5, 3)])
def test_what_records_stand_for_is_quantised_to_itself(d, k_exp, v_exp):
    r = np.random.default_rng(1)
    k, v = r.standard_normal((2, 3, 5, d))
    k[0, 0, 3], v[1, 2, d - 1] = np.nan, np.inf
    rec = Q.quantise(k, v, k_exp, v_exp)
    assert rec.shape == (3, 5, Q.record_size(d))
    rk, rv = Q.dequantise(rec, d, k_exp, v_exp)
    assert np.isnan(rk[0, 0, :16]).all() and np.isnan(rv[1, 2, -16:]).all()
    assert np.isnan(rk).sum() == 16 and np.isnan(rv).sum() == 16
    ok = np.isfinite(k) & ~np.isnan(rk)
    block = np.abs(np.where(np.isfinite(k), k, 0)).reshape(3, 5, -1, 16).max(-1).repeat(16, -1)
    assert np.all((np.abs(rk - k) <= block / 4 + 2.0 ** (k_exp - 10) * 6)[ok])
    again = Q.quantise(rk, rv, k_exp, v_exp)
    same = Q.dequantise(again, d, k_exp, v_exp)
    # The largest of a block may be 4 or 3 steps: another scale then, same values
    # as far as it holds them.
    full = np.abs(rk).reshape(3, 5, -1, 16).max(-1) == 6 * 2.0 ** k_exp * Q.e4m3(rec[..., d:d + d // 16])
    full = full.repeat(16, -1) & ok
    assert np.array_equal(same[0][full], rk[full])


def test_attention_is_the_full_attention_over_what_is_seen():
    r = np.random.default_rng(2)
    q = r.standard_normal((2, 4, 3, 8))
    k, v = r.standard_normal((2, 2, 2, 11, 8))
    kw, vw = r.standard_normal((2, 2, 2, 3, 8))
    o, lse, spread = Q.attention(q, k, v, 0.3, [np.arange(11)] * 2)
    ro, rl = O.full_verify_attention(q, k, v, 0.3)
    np.testing.assert_allclose(o, ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)
    assert np.all(spread >= np.abs(o))
    o, lse, _ = Q.attention(q, k, v, 0.3, [np.array([3]), np.array([], int)])
    assert np.allclose(o[0, 0], v[0, 0, 3]) and not o[1].any() and np.isneginf(lse[1]).all()
    o, lse, _ = Q.attention(q, k, v, 0.3, [[], []], kw, vw)
    assert np.allclose(o[:, 3, 0], vw[:, 1, 0])
    q[0, 0, 0, 0] = np.nan
    o, lse, _ = Q.attention(q, k, v, 0.3, [np.arange(11)] * 2)
    assert np.isnan(lse).sum() == 1 and np.isnan(o[0, 0, 0]).all()


def test_logprobs_closed_forms():
    inf, nan = np.inf, np.nan
    lp, h, lse, ids, best = Q.logprobs(np.zeros(8), 2.0, [3, -1, 8], 3)
    assert np.allclose(lp, [-np.log(8), -inf, -inf]) and np.isclose(h, np.log(8))
    assert np.isclose(lse, np.log(8)) and ids.tolist() == [0, 1, 2] and np.allclose(best, -np.log(8))
    x = np.array([-inf, np.log(0.5), np.log(0.25), np.log(0.25)])
    lp, h, lse, ids, best = Q.logprobs(x, 1.0, [0, 1], 4)
    assert np.isneginf(lp[0]) and np.isclose(lp[1], np.log(0.5)) and np.isclose(h, 1.5 * np.log(2))
    assert ids.tolist() == [1, 2, 3, 0] and np.isneginf(best[3])
    lp, h, lse, ids, best = Q.logprobs(np.full(3, -inf), 1.0, [1], 2)
    assert np.isneginf(lp).all() and h == 0 and np.isneginf(lse) and ids.tolist() == [0, 1]
    for bad in (nan, inf):
        lp, h, lse, ids, best = Q.logprobs(np.array([1.0, bad, 2.0]), 1.0, [0], 3)
        assert np.isnan(lp).all() and np.isnan(h) and np.isnan(lse) and np.isnan(best).all()
        assert ids.tolist() == ([2, 0, -1] if np.isnan(bad) else [1, 2, 0])
