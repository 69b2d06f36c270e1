"""Attention over the 4-bit cache on the GPU, held as a whole to what test_lowbit_accuracy says, in
every way that a call can go."""

import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402
from test_gpu_kv import device  # noqa: E402
from test_lowbit_accuracy import definition, filled, outputs_hold, weights_hold  # noqa: E402

DT = {"f16": (torch.float16, np.float16), "f32": (torch.float32, np.float32)}


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def check(c, q, scale, weights=True):
    """A call's outputs, and its weights, against the definition."""
    dev = device(c)
    x = torch.from_numpy(q).cuda()
    o = torch.empty_like(x)
    w = torch.zeros((q.shape[0], c.H, dev.room), device="cuda") if weights else None
    bcq.bcq_kv_attend(dev, x, o, scale=scale, weights=w)
    ref, total = definition(c, q, float(np.float32(scale)))
    assert outputs_hold(o.cpu().numpy(), ref)
    if weights:
        got = w.cpu().numpy()
        assert weights_hold(got[..., :total.shape[2]], total)
        assert not got[..., total.shape[2]:].any()


# lens, n, heads, cached heads, D, page, pages of a sequence
WAYS = [
    ([120], 1, 8, 2, 128, 16, 8), ([700], 1, 8, 2, 128, 64, 11),  # up to 16 rows; split
    ([700, 450], 2, 8, 2, 64, 64, 11), ([500], 1, 4, 1, 256, 64, 8),
    ([110, 60], 5, 16, 4, 64, 16, 7), ([600], 5, 16, 4, 128, 32, 19),  # up to 32
    ([250], 40, 4, 2, 128, 16, 16), ([200], 70, 4, 2, 64, 16, 13),  # more
    ([200], 40, 4, 2, 256, 16, 13), ([1100], 40, 4, 2, 128, 128, 9),  # more, split
    ([600], 17, 2, 2, 256, 32, 19),
    ([300, 90, 0, 201], 50, 4, 2, 128, 64, 64),  # weights of 64 tokens a workgroup
    ([300, 90, 0, 201], 70, 2, 2, 64, 64, 64),
]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,n,Hq,H,D,page,width", WAYS)
def test_every_way(lens, n, Hq, H, D, page, width, dtype):
    say("kv_attend accuracy", lens, n, Hq, H, D, page, dtype)
    c = filled(lens, H, D, page, width, seed=n + D)
    q = np.random.default_rng(3).normal(size=(len(lens), n, Hq, D)).astype(DT[dtype][1])
    check(c, q, D ** -0.5)
    check(c, q, D ** -0.5, weights=False)


# lens, n, heads, cached heads, D, page, pages of a sequence: few rows, 32, more
FEW = [([300], 1, 8, 2, 128, 64, 5), ([200], 7, 4, 1, 64, 16, 13), ([200], 40, 4, 2, 256, 16, 13)]


@pytest.mark.parametrize("exponent", [-10, -13, -16])
@pytest.mark.parametrize("lens,n,Hq,H,D,page,width", FEW)
def test_small_queries(lens, n, Hq, H, D, page, width, exponent):
    """fp16 queries near and below that type's smallest normal number, with a scale that makes up
    for it."""
    say("kv_attend small queries", lens, n, D, exponent)
    c = filled(lens, H, D, page, width, seed=D)
    q = np.random.default_rng(4).normal(size=(1, n, Hq, D)) * 2.0**exponent
    check(c, q.astype(np.float16), D ** -0.5 * 2.0**-exponent)


@pytest.mark.parametrize("lens,n,Hq,H,D,page,width", FEW)
def test_queries_of_unlike_size(lens, n, Hq, H, D, page, width):
    """Rows of a tile from 1e-5 to 6e4, each with loud and quiet channels."""
    say("kv_attend unlike queries", lens, n, D)
    c = filled(lens, H, D, page, width, seed=D, k_mean=0.1)
    rng = np.random.default_rng(5)
    rows = 2.0 ** rng.integers(-16, 13, (1, n, Hq, 1))
    q = rng.normal(size=(1, n, Hq, D)) * rows * 2.0 ** rng.integers(-4, 1, D)
    check(c, np.clip(q, -6e4, 6e4).astype(np.float16), 1e-3)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 3e7, -1e9, 1e31, -3e33, 3.4e38])
@pytest.mark.parametrize("lens,n,Hq,H,D,page,width", FEW)
def test_scales_up_to_the_largest(lens, n, Hq, H, D, page, width, scale, dtype):
    """Scores of any size: all weight on a row's largest, wherever it lies, shared among equals."""
    say("kv_attend scale", lens, n, D, scale, dtype)
    c = filled(lens, H, D, page, width, seed=1)
    k = np.random.default_rng(7).normal(size=D) * 4
    for t in (2, 3, lens[0] // 2, lens[0] - n):  # the same key, with unlike values
        for h in range(H):
            c.put(0, h, t, k, np.linspace(-1, 1 + t, D))
    q = np.random.default_rng(6).normal(size=(1, n, Hq, D))
    q[0, :, ::2] = k * np.sign(scale)  # half of the heads look for it
    check(c, q.astype(DT[dtype][1]), scale)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_a_million_tokens_in_one_pass(dtype):
    """Values all alike, whose sums grow all the way, for as many rows as leave one workgroup a
    whole sequence: the output is the value."""
    L, n, H, G, D = 1 << 20, 2048 if dtype == "f16" else 512, 8, 4, 128
    say("kv_attend of a million tokens", n, dtype)
    c = bcq.KVCache.new(1, L, H, D, page_tokens=256)
    c.lens.fill_(L)
    k = torch.randn((1, L, 1, D), device="cuda", dtype=torch.float16) * 0.5
    v = torch.randn((1, 1, 1, D), device="cuda")
    bcq.bcq_kv_append(c, k.expand(1, L, H, D), v.half().expand(1, L, H, D))
    value = torch.empty((1, 1, H, D), device="cuda")
    bcq.bcq_kv_read(c, torch.empty_like(value), value)
    q = torch.randn((1, n, H * G, D), device="cuda").to(DT[dtype][0])
    o = torch.empty_like(q)
    bcq.bcq_kv_attend(c, q, o)
    ref = value[0, 0, 0].cpu().numpy().astype(np.float64)
    got = o[0, ::67, ::3].reshape(-1, D).cpu().numpy()
    assert outputs_hold(got, np.broadcast_to(ref, got.shape))
