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
