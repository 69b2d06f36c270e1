"""What attention over the 4-bit cache is held to as a whole, and that this tells its precision
from less (no GPU).

A call's outputs and weights come from scores, sums and products that hold 22 bits and more.
fp32 calls: scores are sums whose terms come to about 30, in roundings of 2^-24 that partly
cancel, so a probability is off by about 1e-6 of itself, and so is the norm of the outputs, which
are averages with those; FP32 and WEIGHTS allow a few times that.  fp16 calls: the output's
own rounding to fp16 is 100 times larger, 2e-4 of the norm; F16 allows as much more as an error of
its own of half that size adds to it (sqrt(1 + 1/4) is 1.12).  Anything held in one fp16 on the
way, 2e-4 of itself, is beyond both."""

import numpy as np
import pytest

from oracle import lowbit as lb

FP32, WEIGHTS, F16 = 2e-6, 4e-6, 1.12


def definition(cache, q, scale):
    """(outputs, summed probabilities) of oracle.lowbit.attend, over whole matrices."""
    q = np.asarray(q).astype(np.float64)
    B, n, Hq, D = q.shape
    G = Hq // cache.H
    out, total = np.zeros_like(q), np.zeros((B, cache.H, int(cache.lens.max(initial=0))))
    for b in range(B):
        L = int(cache.lens[b])
        for h in range(cache.H if L > 0 else 0):
            k, v, _ = cache.get(b, h, np.arange(L))
            x = q[b, :, h * G:(h + 1) * G]
            z = scale * (x @ k.T)
            seen = np.arange(L) <= (L - n + np.arange(n))[:, None, None]
            z = np.where(seen, z, -np.inf)
            top = z.max(axis=-1, keepdims=True)
            p = np.exp(z - np.where(np.isfinite(top), top, 0))
            p /= np.maximum(p.sum(axis=-1, keepdims=True), 1e-300)
            out[b, :, h * G:(h + 1) * G] = p @ v
            total[b, h, :L] = p.sum(axis=(0, 1))
    return out, total


def norm(x):
    return np.linalg.norm(np.asarray(x, np.float64))


def outputs_hold(out, ref):
    """Whether outputs, of their type, are as near the definition's as a call's have to be."""
    if out.dtype == np.float16:
        return norm(out - ref) <= F16 * norm(ref.astype(np.float16) - ref) + FP32 * norm(ref)
    return norm(out - ref) <= FP32 * norm(ref)


def weights_hold(got, total):
    return norm(got - total) <= WEIGHTS * norm(total)


def filled(lens, H, D, page, width, seed, k_mean=1.0):
    rng = np.random.default_rng(seed)
    table = rng.permutation(len(lens) * width).reshape(len(lens), width)
    c = lb.Cache(table.size, H, page, D, table, lens)
    mean = rng.normal(size=(H, D)) * k_mean
    for b, L in enumerate(lens):
        for h in range(H):
            for t, (k, v) in enumerate(rng.normal(size=(L, 2, D))):
                c.put(b, h, t, k + mean[h], v)
    return c


def simulated(cache, q, scale, p_bits=None, q_bits=None):
    """The kernels' way of computing outputs and weights in float64, but for what is held in fewer
    bits: probability times V scale, and the queries (bits of a significand)."""
    def held(x, bits):
        if bits is None:
            return x
        m, e = np.frexp(x)
        return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)

    x = held(np.asarray(q).astype(np.float64), q_bits)
    B, n, Hq, D = x.shape
    out, (_, total) = np.zeros_like(x), definition(cache, x, scale)
    for b in range(B):
        L = int(cache.lens[b])
        for g in range(Hq):
            k, v, s = cache.get(b, g // (Hq // cache.H), np.arange(L))
            code = (v - s[:, 3:4]) / s[:, 2:3]
            for i in range(n):
                m = L - n + i + 1
                z = scale * (k[:m] @ x[b, i, g])
                p = np.exp(z - z.max())
                mid = s[:m, 3] + 7.5 * s[:m, 2]
                out[b, i, g] = (held(p * s[:m, 2], p_bits) @ (code[:m] - 7.5) + p @ mid) / p.sum()
    return out, total


@pytest.mark.parametrize("D,L", [(64, 200), (128, 700), (256, 90)])
def test_the_criterion_tells_one_fp16_from_two(D, L):
    c = filled([L], 2, D, 16, L // 16 + 1, seed=D)
    q = np.random.default_rng(1).normal(size=(1, 3, 4, D))
    for dtype in (np.float16, np.float32):
        x = q.astype(dtype)
        ref, total = definition(c, x, D ** -0.5)
        want, want_total, _, _ = lb.attend(c, x, D ** -0.5)
        assert np.allclose(ref, want, rtol=0, atol=1e-13) and np.allclose(total, want_total)
        out, got = simulated(c, x, D ** -0.5, p_bits=22, q_bits=22)
        assert outputs_hold(out.astype(dtype), ref) and weights_hold(got, total)
        out, _ = simulated(c, x, D ** -0.5, p_bits=11, q_bits=22)
        assert not outputs_hold(out.astype(dtype), ref)
    out, got = simulated(c, x, D ** -0.5, p_bits=22, q_bits=11)  # x in single precision
    assert not outputs_hold(out.astype(np.float32), ref) and not weights_hold(got, total)
