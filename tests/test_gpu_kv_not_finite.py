"""Cached vectors that four bits cannot stand for: what reads them is NaN, and nothing else."""

import sys

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


# smallest and largest value of a vector whose zero, scale or both are past fp16's range
PAST = [(-7e4, -6.9e4), (7e4, 7.1e4), (-6e4, 1e6), (-3e38, 3e38), (1.0, np.inf), (-np.inf, 1.0),
        (-np.inf, np.inf)]


@pytest.mark.parametrize("lo,hi", PAST)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_and_read(D, lo, hi):
    say("kv_append past the range", D, lo, hi)
    x = np.random.default_rng(D).normal(size=(2, 1, 5, 1, D)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        x[0, 0, 1, 0] = np.where(np.arange(D) % 3, lo, hi)
        x[1, 0, 3, 0] = np.where(np.arange(D) % 5, hi, lo)
    c = bcq.KVCache.new(1, 16, 1, D, page_tokens=16)
    c.lens.fill_(5)
    t = torch.from_numpy(x).cuda()
    bcq.bcq_kv_append(c, t[0], t[1])
    want = lb.Cache(1, 1, 16, D, [[0]], [5])
    for i in range(5):
        want.put(0, 0, i, x[0, 0, i, 0], x[1, 0, i, 0])
    assert np.array_equal(c.k_codes.cpu().numpy(), want.k)
    assert np.array_equal(c.v_codes.cpu().numpy(), want.v)
    assert np.array_equal(c.scales.cpu().numpy(), want.s, equal_nan=True)
    got = torch.empty_like(t)
    bcq.bcq_kv_read(c, got[0], got[1])
    nan = torch.isnan(got).all(dim=-1)[:, 0, :, 0].cpu().tolist()
    assert nan == [[i == 1 for i in range(5)], [i == 3 for i in range(5)]]
    assert torch.isfinite(got).all(dim=-1).sum() == 8


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("n", [3, 40])
def test_a_key_past_the_range_is_not_skipped(n, dtype, sign):
    """For queries whose sum has either sign: a score of -inf would hide the token."""
    say("kv_attend key past the range", n, dtype, sign)
    D, L = 64, 100
    x = torch.randn((2, 1, L, 1, D), device="cuda")
    caches = []
    for bad in (False, True):
        if bad:
            x[0, 0, L - 2] = -7e4 + torch.arange(D, device="cuda")
        c = bcq.KVCache.new(1, L, 1, D, page_tokens=16)
        c.lens.fill_(L)
        bcq.bcq_kv_append(c, x[0], x[1])
        caches.append(c)
    q = torch.rand((1, n, 2, D), device="cuda").to(dtype) * sign
    a, b = torch.empty_like(q), torch.empty_like(q)
    for c, o in zip(caches, (a, b)):
        bcq.bcq_kv_attend(c, q, o)
    assert torch.isnan(b[:, -2:]).all()  # the two that see it
    assert torch.equal(a[:, :-2], b[:, :-2]) and torch.isfinite(a).all()


# lens, n, heads, cached heads, D, pages of 16: weights from stored scores, formed again
# one and two tiles of tokens a workgroup
WEIGHTS = [(100, 3, 4, 2, 128, 7), (100, 40, 4, 2, 64, 7), (100, 40, 2, 1, 256, 7),
           (100, 40, 8, 8, 128, 260)]


@pytest.mark.parametrize("part", [2, 3])
@pytest.mark.parametrize("at", ["last", "first", "middle"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("L,n,Hq,H,D,width", WEIGHTS)
def test_weights_do_not_depend_on_values(L, n, Hq, H, D, width, dtype, value, at, part):
    """A V scale or zero that is not finite, in a tile that needs a mask and in one that does not:
    rows that see it have no output and the same weights as ever."""
    say("kv_attend weights beside a bad value", L, n, D, dtype, value, at, part)
    t = {"last": L - n, "first": 0, "middle": 40}[at]
    x = torch.randn((2, 1, L, H, D), device="cuda", generator=torch.Generator("cuda")
                    .manual_seed(1))
    q = torch.randn((1, n, Hq, D), device="cuda").to(dtype)
    got = []
    for bad in (False, True):
        c = bcq.KVCache.new(1, width * 16, H, D, page_tokens=16)
        c.lens.fill_(L)
        bcq.bcq_kv_append(c, x[0], x[1])
        if bad:
            c.scales[t // 16, :, t % 16, part] = value
        o = torch.empty_like(q)
        w = torch.zeros((1, H, c.room), device="cuda")
        bcq.bcq_kv_attend(c, q, o, weights=w)
        got.append((o, w))
    (a, wa), (b, wb) = got
    seen = torch.arange(n, device="cuda") + L - n >= t
    assert not torch.isfinite(b[:, seen]).any() and torch.equal(a[:, ~seen], b[:, ~seen])
    # the reference of the exponentials may differ, and with it the last bits
    assert (wb - wa).norm() <= 4e-6 * wa.norm() and torch.isfinite(wb).all()


@pytest.mark.parametrize("n", [3, 40])
def test_weights_of_a_row_without_any_stay_where_it_sees(n):
    """A query that is NaN leaves nothing on tokens behind it."""
    say("kv_attend weights of a NaN query", n)
    L, D = 70, 64
    x = torch.randn((2, 1, L, 1, D), device="cuda")
    c = bcq.KVCache.new(1, L, 1, D, page_tokens=16)
    c.lens.fill_(L)
    bcq.bcq_kv_append(c, x[0], x[1])
    q = torch.randn((1, n, 2, D), device="cuda")
    o, want = torch.empty_like(q), torch.zeros((1, 1, c.room), device="cuda")
    bcq.bcq_kv_attend(c, q, o, weights=want)
    q[0, n // 2, 0, 5] = float("nan")
    w = torch.zeros_like(want)
    bcq.bcq_kv_attend(c, q, o, weights=w)
    seen = L - n + n // 2 + 1
    assert torch.isnan(w[..., :seen]).all()
    assert torch.equal(w[..., seen:], want[..., seen:])
