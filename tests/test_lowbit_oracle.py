"""The float64 definitions of the low-bit operators against worked values and brute force
(no GPU)."""

import numpy as np
import pytest

from oracle import lowbit as lb


def test_rows_by_hand():
    x = np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [2.54, -2.54, 0.02, 0]], np.float32)
    c, s = lb.quantize_rows(x)
    assert c[0].tolist() == [127, -64, 0, 2] and s[0] == 1  # halves to even
    assert not c[1].any() and s[1] == 0
    assert c[2].tolist() == [127, -127, 1, 0]
    c, s = lb.quantize_rows(np.array([[1, np.inf], [np.nan, 1]], np.float32))
    assert np.isnan(s).all() and not c.any()


def test_product_by_hand():
    y = lb.product(np.array([[1, -2]], np.int8), np.array([0.5], np.float32),
                   np.array([[3, 4], [-128, 127]], np.int8), np.array([2, 1], np.float32),
                   np.array([1, 0], np.float32))
    assert y.tolist() == [[1 * (3 - 8) + 1, 0.5 * (-128 - 254)]]


def test_vectors_by_hand():
    c, s, z = lb.quantize_vectors(np.array([[-1, 0, 0.5, 14], [3, 3, 3, 3]], np.float32))
    assert (s[0], z[0]) == (1, -1) and c[0].tolist() == [0, 1, 2, 15]  # 1.5 rounds to 2
    assert (s[1], z[1]) == (0, 3) and not c[1].any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_hold_what_is_put(D):
    rng = np.random.default_rng(D)
    c = lb.Cache(5, 2, 16, D, [[3, 0], [4, 1]], [29, 7])
    want = {}
    for b, n in ((0, 29), (1, 7)):
        for h in range(2):
            for t in rng.permutation(n):
                k, v = rng.normal(size=(2, D)).astype(np.float32)
                c.put(b, h, int(t), k, v)
                want[b, h, int(t)] = (k, v)
    for (b, h, t), (k, v) in want.items():
        gk, gv, s = c.get(b, h, [t])
        for got, x, step in ((gk, k, s[0, 0]), (gv, v, s[0, 2])):
            # half a step, and what the fp16 zero and scale are off by
            assert np.abs(got[0] - x).max() <= step * 0.5 + 2.0**-10 * np.abs(x).max() * 2
    byte, shift = lb.v_place(D)
    at = {(int(x) + 2 * t, int(y)) for x, y in zip(byte, shift) for t in range(4)}
    assert len(at) == 4 * D and max(a for a, _ in at) == 2 * D - 1  # a bijection onto the block


def test_attention_against_a_loop():
    rng = np.random.default_rng(3)
    c = lb.Cache(4, 1, 16, 64, [[2, 1]], [19])
    for t in range(19):
        c.put(0, 0, t, *rng.normal(size=(2, 64)))
    q = rng.normal(size=(1, 2, 2, 64))
    out, total, _, _ = lb.attend(c, q, 0.125)
    k, v, _ = c.get(0, 0, np.arange(19))
    seen = np.zeros(19)
    for i in range(2):
        for g in range(2):
            m = 18 + i
            e = [np.exp(0.125 * sum(q[0, i, g, d] * k[t, d] for d in range(64))) for t in range(m)]
            o = sum(e[t] * v[t] for t in range(m)) / sum(e)
            assert np.allclose(out[0, i, g], o, rtol=1e-12, atol=1e-12)
            seen[:m] += np.array(e) / sum(e)
    assert np.allclose(total[0, 0], seen)


def test_queries_before_the_cache_see_nothing():
    c = lb.Cache(1, 1, 16, 64, [[0]], [1])
    c.put(0, 0, 0, np.ones(64), np.arange(64.0))
    out, total, _, _ = lb.attend(c, np.ones((1, 3, 1, 64)), 1.0)
    assert not out[0, :2].any() and out[0, 2].any() and total[0, 0, 0] == 1


def test_eviction_by_hand():
    w = np.array([5, 1, 4, 1, 9, 1, 0], np.float32)
    pos = np.arange(7)
    assert lb.kept_slots(7, 4, 1, w, pos).tolist() == [0, 2, 4, 6]
    # slots 0, 2 stay, the evicted 1 and 3 take 4 and 6
    assert lb.evict(7, 4, 1, w, pos).tolist() == [0, 4, 2, 6]
    assert lb.kept_slots(7, 5, 0, w, pos).tolist() == [0, 1, 2, 3, 4]  # ties: the lower slots
    assert lb.evict(3, 4, 1, w, pos).tolist() == [0, 1, 2]
    assert lb.kept_slots(3, 2, 0, np.array([np.nan, -np.inf, 0], np.float32), pos).tolist() == [1, 2]


def test_vectors_past_the_range_have_no_scale():
    x = np.array([[-7e4, -6.9e4], [7e4, 7e4], [1, np.inf], [-np.inf, 1], [np.nan, 1],
                  [-6e4, 1e6], [0, 9e5]], np.float32)
    c, s, _ = lb.quantize_vectors(x)
    assert np.isnan(s[:6]).all() and not c[:6].any() and np.isfinite(s[6]) and c[6, 1] == 15
