"""The attention block's oracle against hand-derived values, closed forms and reductions.
CPU only."""
import math

import numpy as np
import pytest

from oracle import attention as OA


def test_rope_hand_values():
    # one pair, a quarter turn: (1, 0) -> (0, 1), (0, 1) -> (-1, 0); position 0 leaves x alone
    inv = [math.pi / 2]
    x = np.array([[[1.0, 0.0, 7.0]], [[1.0, 0.0, 7.0]], [[0.0, 1.0, 7.0]]])
    y = OA.rope(x, [[0, 1, 1]], inv)
    assert np.allclose(y[:, 0], [[1, 0, 7], [0, 1, 7], [-1, 0, 7]], atol=1e-15)


def test_rope_pairing_and_axes():
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    half = OA.rope(x, [[1], [0]], [math.pi / 2, math.pi / 2], axis=[0, 1])
    assert np.allclose(half, [[[-3, 2, 1, 4]]])          # pair (1, 3) turned, (2, 4) at position 0
    inter = OA.rope(x, [[1], [0]], [math.pi / 2, math.pi / 2], axis=[0, 1], interleaved=True)
    assert np.allclose(inter, [[[-2, 1, 3, 4]]])


def test_rope_keeps_relative_positions():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 8))
    inv = 100.0 ** (-np.arange(4) / 4)
    dots = [float((OA.rope(q, [[a]], inv) * OA.rope(k, [[a + 5]], inv)).sum()) for a in (0, 3, 1000)]
    assert np.ptp(dots) < 1e-9 and abs(np.linalg.norm(OA.rope(q, [[77]], inv)) - np.linalg.norm(q)) < 1e-12


@pytest.mark.parametrize("amax,e", [(127.0, 0), (127.5, 1), (63.5, -1), (63.51, 0), (1.0, -6), (0.0, -126),
                                    (1e-45, -126), (2.0 ** -119 * 127 / 128, -126), (2.0 ** -119, -125),
                                    (3.3895313892515355e38, 122)])
def test_page_exponent(amax, e):
    assert OA.page_exponent(amax) == e
    assert amax <= math.ldexp(127, e) and (e == -126 or amax > math.ldexp(127, e - 1))


def test_cache_hand_values():
    c = OA.PagedCache(2, 4, 1, 2)
    one = lambda a, b: np.array([[[a, b]]], dtype=float)
    c.write([1], 0, one(3.0, -127.0), one(0.5, 0.0))      # e = 0; e = -7: 0.5 = 64 * 2^-7
    assert c.e["k"][1, 0] == 0 and c.q["k"][1, 0, 0].tolist() == [3, -127]
    assert c.e["v"][1, 0] == -7 and c.q["v"][1, 0, 0].tolist() == [64, 0]
    c.write([1], 1, one(254.0, 5.0), one(0.25, 0.25))     # e = 1: 3 -> 1.5 -> 2, -127 -> -63.5 -> -64, 5 -> 2.5 -> 2
    assert c.e["k"][1, 0] == 1 and c.q["k"][1, :2, 0].tolist() == [[2, -64], [127, 2]]
    assert c.e["v"][1, 0] == -7 and c.q["v"][1, 1, 0].tolist() == [32, 32]
    k, v = c.read([1], 0, 2)
    assert k[:, 0].tolist() == [[4, -128], [254, 4]] and v[:, 0].tolist() == [[0.5, 0], [0.25, 0.25]]
    c.write([1], 0, one(1.0, 1.0), one(1.0, 1.0))         # slot 0: the page starts anew
    assert c.e["k"][1, 0] == -6 and c.q["k"][1, 0, 0].tolist() == [64, 64]
    c.write([1], 2, one(math.nan, 0.0), one(math.inf, 0.0))
    assert all(np.isnan(t).all() for t in c.read([1], 0, 3))
    c.write([9], 0, one(1.0, 1.0), one(1.0, 1.0))         # outside the pool: nothing happens
    assert np.isnan(c.read([9], 0, 1)[0]).all()


def test_cache_error_stays_below_one_step_however_often_a_scale_grows():
    rng = np.random.default_rng(1)
    T = 16
    c = OA.PagedCache(1, T, 1, 8)
    x = rng.standard_normal((T, 1, 8)) * (1.7 ** np.arange(T))[:, None, None]   # grows at most tokens
    for t in range(T):
        c.write([0], t, x[t:t + 1], x[t:t + 1])
    got, _ = c.read([0], 0, T)
    assert np.max(np.abs(got - x)) < math.ldexp(1.0, int(c.e["k"][0, 0]))


def test_attend_closed_forms():
    # equal scores: the mean of what a row sees
    k = np.zeros((5, 1, 2))
    v = np.arange(5.0).reshape(5, 1, 1) * np.ones((1, 1, 2))
    q = np.ones((3, 2, 2))
    out, lse, mass, size = OA.attend(q, k, v, 1.0)
    assert np.allclose(out[:, 0, 0], [1.0, 1.5, 2.0]) and np.allclose(lse[:, 1], np.log([3, 4, 5]))
    out, _, _, _ = OA.attend(q, k, v, 1.0, window=2)
    assert np.allclose(out[:, 0, 0], [1.5, 2.5, 3.5])
    out, _, _, _ = OA.attend(q, k, v, 1.0, causal=False)
    assert np.allclose(out, 2.0)
    # ln 3 apart: weights 1/4 and 3/4
    out, lse, _, _ = OA.attend(np.ones((1, 1, 1)), np.array([[[0.0]], [[math.log(3)]]]), np.array([[[0.0]], [[4.0]]]), 1.0)
    assert np.allclose(out, 3.0) and np.allclose(lse, math.log(4))


def test_attend_rows_that_see_nothing():
    q = np.ones((4, 1, 2))
    out, lse, _, _ = OA.attend(q, np.ones((2, 1, 2)), np.ones((2, 1, 2)), 1.0)  # positions -2, -1, 0, 1
    assert out[:2].tolist() == np.zeros((2, 1, 2)).tolist() and np.isneginf(lse[:2]).all()
    assert np.allclose(out[2:], 1.0)
    out, lse, _, _ = OA.attend(q, np.ones((0, 1, 2)), np.ones((0, 1, 2)), 1.0, causal=False)
    assert not out.any() and np.isneginf(lse).all()


def test_attend_shares_key_heads():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((2, 6, 4)), rng.standard_normal((7, 2, 4)), rng.standard_normal((7, 2, 4))
    out, *_ = OA.attend(q, k, v, 0.5)
    for h in range(6):
        one, *_ = OA.attend(q[:, h:h + 1], k[:, h // 3:h // 3 + 1], v[:, h // 3:h // 3 + 1], 0.5)
        assert np.allclose(out[:, h], one[:, 0])


def test_planted_mistakes_are_caught(monkeypatch):
    """Each plausible mistake makes one of the checks above fail."""
    def fails(check, *args):
        try:
            check(*args)
        except AssertionError:
            return True
        return False

    with monkeypatch.context() as mp:      # half away from zero instead of to even
        mp.setattr(OA.np, "rint", lambda a: np.sign(a) * np.floor(np.abs(a) + 0.5))
        assert fails(test_cache_hand_values)
    with monkeypatch.context() as mp:      # scale = next power of two of the maximum
        mp.setattr(OA, "page_exponent", lambda a: OA.POISON if not math.isfinite(a) else math.frexp(a)[1] - 7)
        assert fails(test_page_exponent, 127.5, 1)
    real = OA.attend
    with monkeypatch.context() as mp:      # the window one key too long
        mp.setattr(OA, "attend", lambda *a, window=0, **k: real(*a, window=window + 1 if window else 0, **k))
        assert fails(test_attend_closed_forms)
    turn = OA.rope
    with monkeypatch.context() as mp:      # turned the other way
        mp.setattr(OA, "rope", lambda x, p, f, **k: turn(x, -np.asarray(p), f, **k))
        assert fails(test_rope_hand_values) and fails(test_rope_pairing_and_axes)
