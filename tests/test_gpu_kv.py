"""The 4-bit key/value cache on the GPU: append, read, attention and eviction against their
float64 definitions.  What is quantized, moved or chosen is compared to the bit; attention within
what its roundings allow (see bound)."""

import math
import sys

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402

DT = {"f16": (torch.float16, np.float16), "f32": (torch.float32, np.float32)}


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def make(lens, H, D, page, width, seed=0, k_mean=1.0, v_scale=None):
    """A host cache of random vectors in shuffled pages, entries past the lengths naming none and
    unused slots holding NaN scales."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    pages = B * width + 2
    table = rng.permutation(pages)[:B * width].reshape(B, width)
    c = lb.Cache(pages, H, page, D, table, lens)
    c.k[:] = rng.integers(0, 256, c.k.shape)
    c.v[:] = rng.integers(0, 256, c.v.shape)
    c.s[:] = np.nan
    mean = rng.normal(size=(H, D)) * k_mean
    for b in range(B):
        for h in range(H):
            for t in range(int(lens[b])):
                k = rng.normal(size=D) + mean[h]
                v = rng.normal(size=D) + 0.3
                if v_scale is not None:
                    v = v * v_scale(t)
                c.put(b, h, t, k.astype(np.float32), v.astype(np.float32))
    for b in range(B):
        c.table[b, (max(int(lens[b]), 0) + page - 1) // page:] = [-1, 1 << 30][b % 2]
    return c


def device(c):
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return bcq.KVCache(up(c.k), up(c.v), up(c.s), up(c.table), up(c.lens))


def bound(ref, b, D, T, dtype):
    """|error| of attention's outputs.  Scores: sums of D products and a few more operations in
    fp32, whose relative errors the probabilities take over twice (in the sum too).  Sums over T
    tokens in fp32.  Probability times V scale: one rounding of 2^-11 in fp16 calls, 2^-21 in fp32
    calls, and at most 2^-24 of the row's largest where it is below fp16's normal range.  The
    output's own rounding."""
    score = 2 * (2 * D) * 2.0**-24 * b[0]
    sums = (T + 16) * 2.0**-23 * (b[1] + np.abs(ref))
    p = (2.0**-11 if dtype == "f16" else 2.0**-21) * b[1] + 2.0**-24 * b[2]
    last = 2.0**-11 * np.abs(ref) + 2.0**-24 if dtype == "f16" else 2.0**-23 * np.abs(ref)
    return score + sums + p + last


# lens, n, heads, cached heads, D, page
ATTEND = [
    ([1], 1, 1, 1, 64, 16),
    ([0, 3], 1, 2, 2, 64, 16),
    ([15, 16, 17], 1, 4, 2, 128, 16),
    ([31, 32, 33, 64], 1, 8, 1, 128, 32),
    ([130, 5], 1, 14, 2, 128, 64),
    ([300], 1, 32, 8, 128, 64),
    ([77, 200], 1, 16, 1, 256, 32),
    ([65], 2, 8, 8, 64, 128),
    ([100, 3, 0], 5, 4, 2, 64, 16),
    ([257], 5, 14, 2, 128, 64),  # 35 rows
    ([90], 4, 8, 1, 128, 16),  # 32 rows
    ([40, 20], 17, 2, 2, 256, 16),  # 17 rows of 256 channels
    ([70, 33], 33, 2, 1, 128, 32),
    ([150, 129], 130, 2, 2, 64, 256),
    ([50, 140], 70, 7, 1, 128, 16),
    ([20], 29, 3, 1, 64, 16),  # more queries than tokens
    ([1500], 3, 2, 1, 64, 64),
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,n,Hq,H,D,page", ATTEND)
def test_attend(lens, n, Hq, H, D, page, dtype, weights):
    say("kv_attend", lens, n, Hq, H, D, page, dtype, weights)
    width = (max(lens) + page - 1) // page + 1
    c = make(lens, H, D, page, width, seed=n + D)
    dev = device(c)
    rng = np.random.default_rng(1)
    q = rng.normal(size=(len(lens), n, Hq, D)).astype(DT[dtype][1])
    o = torch.full(q.shape, 7.0, dtype=DT[dtype][0], device="cuda")
    w = torch.full((len(lens), H, dev.room), 0.25, device="cuda") if weights else None
    scale = 1 / math.sqrt(D)
    bcq.bcq_kv_attend(dev, torch.from_numpy(q).cuda(), o, weights=w)
    torch.cuda.synchronize()
    ref, total, b, wb = lb.attend(c, q, np.float32(scale))
    err = np.abs(o.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(ref, b, D, max(lens), dtype)).all()
    if weights:
        T = total.shape[2]
        got = w.cpu().numpy().astype(np.float64)
        tol = 4 * D * 2.0**-24 * 2 * wb + (T + n * Hq + 16) * 2.0**-23 * (total + 0.25)
        assert (np.abs(got[..., :T] - 0.25 - total) <= tol).all()
        for i, L in enumerate(lens):
            assert (got[i, :, L:] == 0.25).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n,Hq,D", [(40, 8, 64), (19, 16, 128), (9, 16, 256)])
def test_attend_weights_of_many_rows_in_a_large_cache(n, Hq, D, dtype):
    """Room for far more tokens than there are: the weights' workgroups take several tiles each."""
    lens, H, page, width = [70, 33, 0, 129], 8, 16, 65
    say("kv_attend weights", n, Hq, D, dtype)
    c = make(lens, H, D, page, width, seed=n)
    dev = device(c)
    q = np.random.default_rng(2).normal(size=(4, n, Hq, D)).astype(DT[dtype][1])
    o = torch.empty(q.shape, dtype=DT[dtype][0], device="cuda")
    w = torch.full((4, H, dev.room), 0.25, device="cuda")
    bcq.bcq_kv_attend(dev, torch.from_numpy(q).cuda(), o, weights=w)
    ref, total, b, wb = lb.attend(c, q, np.float32(1 / math.sqrt(D)))
    err = np.abs(o.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(ref, b, D, max(lens), dtype)).all()
    got = w.cpu().numpy().astype(np.float64)
    T = total.shape[2]
    tol = 4 * D * 2.0**-24 * 2 * wb + (T + n * Hq + 16) * 2.0**-23 * (total + 0.25)
    assert (np.abs(got[..., :T] - 0.25 - total) <= tol).all()
    for i, L in enumerate(lens):
        assert (got[i, :, L:] == 0.25).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("spread", [1e-4, 1e3, None])
def test_attend_v_scales_of_any_size(spread, dtype):
    """Values all tiny, all large, or from 1e-3 to 1e3 within a row."""
    scale_of = (lambda t: spread) if spread else (lambda t: 10.0 ** (t % 7 - 3))
    c = make([150], 1, 128, 16, 10, seed=5, v_scale=scale_of)
    dev = device(c)
    q = np.random.default_rng(2).normal(size=(1, 1, 4, 128)).astype(DT[dtype][1])
    o = torch.empty(q.shape, dtype=DT[dtype][0], device="cuda")
    bcq.bcq_kv_attend(dev, torch.from_numpy(q).cuda(), o)
    ref, _, b, _ = lb.attend(c, q, np.float32(1 / math.sqrt(128)))
    err = np.abs(o.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(ref, b, 128, 150, dtype)).all()


@pytest.mark.parametrize("n", [1, 40])
def test_attend_sharp_softmax(n):
    """Scores hundreds apart, the largest first and last: sums are rescaled on the way."""
    D, L = 64, 200
    c = make([L], 1, D, 16, 13, seed=6)
    for t in (0, 100, L - n):
        c.put(0, 0, t, np.linspace(1, 2, D) * (3 + t / 20), np.linspace(-1, 1, D))
    dev = device(c)
    q = np.full((1, n, 2, D), 4.0, np.float32)
    o = torch.empty(q.shape, device="cuda")
    w = torch.zeros((1, 1, dev.room), device="cuda")
    bcq.bcq_kv_attend(dev, torch.from_numpy(q).cuda(), o, weights=w, scale=1.0)
    ref, total, b, wb = lb.attend(c, q, 1.0)
    err = np.abs(o.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(ref, b, D, L, "f32")).all()
    assert (np.abs(w.cpu().numpy()[..., :L] - total) <= 8 * D * 2.0**-24 * wb
            + (L + 2 * n + 16) * 2.0**-23 * total).all()


@pytest.mark.parametrize("scale", [-0.2, 0.0, -0.0, 1e-30])
@pytest.mark.parametrize("n,dtype", [(1, "f16"), (1, "f32"), (40, "f16")])
def test_attend_scales_of_either_sign(n, dtype, scale):
    c = make([190], 1, 64, 32, 7, seed=3)
    dev = device(c)
    q = np.random.default_rng(4).normal(size=(1, n, 2, 64)).astype(DT[dtype][1])
    o = torch.empty(q.shape, dtype=DT[dtype][0], device="cuda")
    w = torch.zeros((1, 1, dev.room), device="cuda")
    bcq.bcq_kv_attend(dev, torch.from_numpy(q).cuda(), o, scale=scale, weights=w)
    ref, total, b, wb = lb.attend(c, q, np.float32(scale))
    err = np.abs(o.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(ref, b, 64, 190, dtype)).all()
    tol = 4 * 64 * 2.0**-24 * 2 * wb + (190 + n * 2 + 16) * 2.0**-23 * total
    assert (np.abs(w.cpu().numpy()[..., :190].astype(np.float64) - total) <= tol).all()


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("n,dtype", [(2, "f16"), (2, "f32"), (40, "f16"), (40, "f32")])
def test_queries_that_are_not_finite_stay_alone(n, dtype, value):
    c = make([90], 1, 64, 16, 6, seed=5)
    q = np.random.default_rng(6).normal(size=(1, n, 2, 64)).astype(DT[dtype][1])
    ref, _, b, _ = lb.attend(c, q, np.float32(0.125))
    q[0, n // 2, 1, 7] = value
    o = torch.empty(q.shape, dtype=DT[dtype][0], device="cuda")
    bcq.bcq_kv_attend(device(c), torch.from_numpy(q).cuda(), o)
    got = o.cpu().numpy().astype(np.float64)
    assert np.isnan(got[0, n // 2, 1]).all()
    got[0, n // 2, 1] = ref[0, n // 2, 1]
    assert (np.abs(got - ref) <= bound(ref, b, 64, 90, dtype)).all()


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("n", [3, 40])
def test_hidden_tokens_do_not_reach_earlier_queries(n, value):
    D, L = 128, 100
    c = make([L], 2, D, 32, 4, seed=7)
    clean = device(c)
    p, line = c.table[0, (L - 1) // 32], (L - 1) % 32
    c.s[p, :, line] = value
    bad = device(c)
    q = torch.randn((1, n, 4, D), device="cuda", dtype=torch.float16)
    a, b = torch.empty_like(q), torch.empty_like(q)
    wa, wb = (torch.zeros((1, 2, clean.room), device="cuda") for _ in range(2))
    bcq.bcq_kv_attend(clean, q, a, weights=wa)
    bcq.bcq_kv_attend(bad, q, b, weights=wb)
    assert torch.equal(a[:, :-1], b[:, :-1])
    assert not torch.isfinite(b[:, -1]).any()


def test_attend_strides_and_page_order():
    """Queries as a slice of a fused projection, outputs head-major, pages in another order."""
    D, H, L = 64, 2, 70
    c = make([L, 40], H, D, 16, 6, seed=8)
    dev = device(c)
    qkv = torch.randn((2, 3, 3 * H * 2, D), device="cuda")
    q = qkv[:, :, H:3 * H]
    o = torch.full((2, 2 * H, 3, D + 1), 7.0, device="cuda")
    out = o[..., 1:].transpose(1, 2)  # element aligned only
    bcq.bcq_kv_attend(dev, q, out)
    plain = torch.empty((2, 3, 2 * H, D), device="cuda")
    bcq.bcq_kv_attend(dev, q.contiguous(), plain)
    assert torch.equal(out, plain) and (o[..., 0] == 7).all()
    odd = torch.empty((2, 3, 2 * H, D + 3), device="cuda")[..., 3:]
    odd.copy_(q)
    bcq.bcq_kv_attend(dev, odd, plain)
    assert torch.equal(out, plain)
    # pages elsewhere, the same tokens
    perm = np.random.default_rng(1).permutation(c.k.shape[0])
    inv = np.argsort(perm)
    moved = lb.Cache(c.k.shape[0], H, 16, D, c.table, c.lens)
    moved.k, moved.v, moved.s = c.k[perm], c.v[perm], c.s[perm]
    ok = (c.table >= 0) & (c.table < len(perm))
    moved.table = np.where(ok, inv[np.where(ok, c.table, 0)], c.table).astype(np.int32)
    bcq.bcq_kv_attend(device(moved), q, plain)
    assert torch.equal(out, plain)


def test_long_cache_past_four_gigabytes():
    """Codes past the reach of 32-bit offsets, at both ends of the pool."""
    H, D, page = 8, 128, 256
    pages = (5 << 30) // (H * page * D // 2)
    k = torch.empty((pages, H, page, D // 2), dtype=torch.uint8, device="cuda")
    v = torch.empty((pages, H, page // 4, 2 * D), dtype=torch.uint8, device="cuda")
    s = torch.empty((pages, H, page, 4), dtype=torch.float16, device="cuda")
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([400], dtype=torch.int32, device="cuda")
    big = bcq.KVCache(k, v, s, table, lens)
    small = bcq.KVCache.new(1, 512, H, D, page_tokens=page)
    small.lens.fill_(400)
    x = torch.randn((2, 1, 400, H, D), device="cuda")
    for c in (big, small):
        bcq.bcq_kv_append(c, x[0], x[1])
    q = torch.randn((1, 1, 8, D), device="cuda")
    out = []
    for c in (big, small):
        o, r = torch.empty_like(q), torch.empty_like(x)
        bcq.bcq_kv_attend(c, q, o)
        bcq.bcq_kv_read(c, r[0], r[1])
        w, pos = c.tracking()
        w.uniform_()
        w.copy_(torch.arange(w.shape[2], device="cuda") % 13)
        pos.copy_(torch.arange(w.shape[2], device="cuda"))
        c.lens.fill_(400)
        bcq.bcq_kv_evict(c, 300, 5, w, pos)
        e = torch.empty_like(q)
        bcq.bcq_kv_attend(c, q, e)
        out.append((o, r, e, c.lens.clone(), pos[..., :300].clone()))
    for a, b in zip(*out):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------ append, read


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,n,H,D,page", [
    ([1], 1, 1, 64, 16), ([5, 0, 2], 3, 2, 64, 16), ([64, 63], 1, 8, 128, 64),
    ([40, 17], 17, 3, 128, 16), ([33], 33, 2, 256, 32), ([300, 256], 256, 1, 128, 256)])
def test_append_and_read(lens, n, H, D, page, dtype):
    say("kv_append", lens, n, H, D, page, dtype)
    rng = np.random.default_rng(n + D)
    width = (max(lens) + page - 1) // page + 1
    c = make([0] * len(lens), H, D, page, width)
    c.table = rng.permutation(len(lens) * width + 2)[:len(lens) * width].reshape(len(lens), width)
    c.table = c.table.astype(np.int32)
    c.lens = np.array(lens, np.int32)
    dev = device(c)
    x = rng.normal(size=(2, len(lens), n, H, D)) * 10.0 ** rng.integers(-2, 3, (2, 1, n, H, 1))
    x = x.astype(DT[dtype][1])
    x[0, 0, 0, 0] = 2.5  # a constant vector
    t = torch.from_numpy(x).cuda()
    w, pos = dev.tracking()
    w += 9
    positions = torch.arange(len(lens) * n, dtype=torch.int32, device="cuda").view(-1, n)
    bcq.bcq_kv_append(dev, t[0], t[1], positions=positions, weights=w, pos=pos)
    want_w, want_pos = np.full(w.shape, 9.0), np.zeros(pos.shape)
    for b, L in enumerate(lens):
        for i in range(n):
            if L - n + i >= 0:
                want_w[b, :, L - n + i], want_pos[b, :, L - n + i] = 0, b * n + i
                for h in range(H):
                    c.put(b, h, L - n + i, x[0, b, i, h], x[1, b, i, h])
    assert np.array_equal(dev.k_codes.cpu().numpy(), c.k)
    assert np.array_equal(dev.v_codes.cpu().numpy(), c.v)
    assert np.array_equal(dev.scales.cpu().numpy(), c.s, equal_nan=True)
    assert np.array_equal(w.cpu().numpy(), want_w) and np.array_equal(pos.cpu().numpy(), want_pos)
    got = torch.full(x.shape, 7.0, dtype=DT[dtype][0], device="cuda")
    bcq.bcq_kv_read(dev, got[0], got[1])
    ref = np.zeros(x.shape)
    for b, L in enumerate(lens):
        i = np.arange(max(0, n - L), n)
        for h in range(H):
            if len(i):
                k, v, _ = c.get(b, h, L - n + i)
                ref[0, b, i, h], ref[1, b, i, h] = k, v
    # zero + scale * code in fp32 (one product, one sum), rounded once
    tol = 2.0**-23 * np.abs(ref).max() + (2.0**-11 * np.abs(ref) if dtype == "f16" else 0)
    assert (np.abs(got.cpu().numpy() - ref) <= tol).all()


def test_append_strided_matches_contiguous():
    H, D = 2, 128
    for off in (0, 1):  # aligned for wide loads, and not
        base = torch.randn((2, 5, 3 * H, D + 4), device="cuda").half()
        k, v = base[:, :, :H, off:off + D], base[:, :, 2 * H:, off:off + D]
        a, b = (bcq.KVCache.new(2, 32, H, D, page_tokens=16) for _ in range(2))
        for c, x, y in ((a, k, v), (b, k.contiguous(), v.contiguous())):
            c.lens.fill_(9)
            bcq.bcq_kv_append(c, x, y)
            assert c.scales.any()
        assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)
        assert torch.equal(a.scales, b.scales)


def test_append_what_is_not_finite():
    c = bcq.KVCache.new(1, 16, 1, 64, page_tokens=16)
    c.lens.fill_(3)
    k = torch.randn((1, 3, 1, 64), device="cuda")
    k[0, 1, 0, 5] = float("nan")
    v = torch.randn((1, 3, 1, 64), device="cuda")
    bcq.bcq_kv_append(c, k, v)
    r = torch.empty_like(k), torch.empty_like(v)
    bcq.bcq_kv_read(c, *r)
    assert torch.isnan(r[0][0, 1]).all() and torch.isfinite(r[0][0, [0, 2]]).all()
    assert torch.isfinite(r[1]).all()


def test_entries_that_name_no_page_are_not_followed():
    c = bcq.KVCache.new(2, 32, 1, 64, page_tokens=16)
    c.page_table[1] = torch.tensor([-5, 99], dtype=torch.int32)
    c.lens.fill_(20)
    x = torch.randn((2, 2, 20, 1, 64), device="cuda")
    before = c.k_codes.clone()
    bcq.bcq_kv_append(c, x[0], x[1])
    assert torch.equal(c.k_codes[2:], before[2:])  # sequence 1's pages were never named
    r = torch.empty_like(x)
    bcq.bcq_kv_read(c, r[0], r[1])
    assert not r[:, 1].any() and r[:, 0].any()
    q = torch.randn((2, 1, 1, 64), device="cuda")
    o = torch.empty_like(q)
    w, pos = c.tracking()
    bcq.bcq_kv_attend(c, q, o, weights=w)
    bcq.bcq_kv_evict(c, 7, 2, w, pos)
    torch.cuda.synchronize()
    assert c.lens.tolist() == [7, 7]


# ------------------------------------------------------------------------------ eviction


EVICT = [  # lens, keep, recent, heads, D, page, room
    ([5], 3, 1, 1, 64, 16, 16), ([10, 3, 0, 4], 4, 2, 2, 64, 16, 16),
    ([65, 64, 66], 64, 10, 2, 128, 32, 96), ([200], 1, 0, 1, 128, 16, 208),
    ([200, 199], 150, 150, 1, 256, 64, 256), ([1500, 700], 333, 20, 2, 64, 64, 1536),
    ([33000, 1030], 1027, 100, 1, 64, 256, 33024), ([90], 1000, 5, 1, 64, 16, 96)]


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,keep,recent,H,D,page,room", EVICT)
def test_evict(lens, keep, recent, H, D, page, room, kind):
    say("kv_evict", lens, keep, recent, H, D, page, room, kind)
    rng = np.random.default_rng(len(lens) + keep)
    B, width = len(lens), room // page
    pages = B * width
    table = rng.permutation(pages).reshape(B, width).astype(np.int32)
    c = lb.Cache(pages, H, page, D, table, np.array(lens, np.int32))
    c.k[:] = rng.integers(0, 256, c.k.shape)
    c.v[:] = rng.integers(0, 256, c.v.shape)
    c.s[:] = rng.normal(size=c.s.shape)
    w = {"spread": lambda: np.exp(2 * rng.normal(size=(B, H, room))),
         "ties": lambda: rng.integers(0, 4, (B, H, room)) * 0.5,
         "odd": lambda: rng.choice([0.0, -0.0, -1.5, 1e-40, np.inf, -np.inf, np.nan, 3.0],
                                   (B, H, room))}[kind]().astype(np.float32)
    pos = np.stack([[rng.permutation(room) for _ in range(H)] for _ in range(B)]).astype(np.int32)
    dev = device(c)
    wd, pd = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    wo, po = torch.full_like(wd, 7), torch.full_like(pd, 7)
    lo = torch.zeros(B, dtype=torch.int32, device="cuda")
    bcq.bcq_kv_evict(dev, keep, recent, wd, pd, lens_out=lo, weights_out=wo, pos_out=po)
    assert lo.tolist() == [min(L, keep) for L in lens] and dev.lens.tolist() == list(lens)
    assert np.array_equal(wd.cpu().numpy(), w, equal_nan=True)
    k, v, s = (t.cpu().numpy() for t in (dev.k_codes, dev.v_codes, dev.scales))
    after = lb.Cache(pages, H, page, D, table, c.lens)
    after.k, after.v, after.s = k, v, s
    for b, L in enumerate(lens):
        for h in range(H):
            src = lb.evict(L, keep, recent, w[b, h], pos[b, h])
            m = len(src)
            assert np.array_equal(wo[b, h, :m].cpu().numpy(), w[b, h, src], equal_nan=True)
            assert np.array_equal(po[b, h, :m].cpu().numpy(), pos[b, h, src])
            assert (wo[b, h, m:] == 7).all() and (po[b, h, m:] == 7).all()
            for got, want in zip(after.get(b, h, np.arange(m)), c.get(b, h, src)):
                assert np.array_equal(got, want)
    # in place, from the same start
    dev = device(c)
    bcq.bcq_kv_evict(dev, keep, recent, wd, pd)
    assert torch.equal(dev.lens, lo)
    assert np.array_equal(dev.k_codes.cpu().numpy(), k)
    assert np.array_equal(dev.v_codes.cpu().numpy(), v)
    assert np.array_equal(dev.scales.cpu().numpy(), s)
    for b, L in enumerate(lens):
        m = min(L, keep)
        assert np.array_equal(wd[b, :, :m].cpu().numpy(), wo[b, :, :m].cpu().numpy(),
                              equal_nan=True)
        assert torch.equal(pd[b, :, :m], po[b, :, :m])


# evictions of one to four tokens, moves made by the selecting workgroup at every number of
# channels, more equal weights than are listed
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,keep,recent,H,D,page,room", [
    ([68, 67], 64, 10, 2, 64, 16, 80), ([5003], 5000, 9, 1, 64, 64, 5056),
    ([250], 200, 10, 1, 256, 64, 256), ([5056, 5030], 5000, 40, 1, 128, 32, 5056),
    ([5002, 5001], 5000, 9, 1, 64, 64, 5056), ([33002], 33000, 7, 1, 64, 256, 33024),
    ([5056], 1000, 100, 1, 64, 64, 5056), ([33024], 33020, 7, 1, 64, 256, 33024)])
def test_evict_by_way(lens, keep, recent, H, D, page, room, kind):
    test_evict(lens, keep, recent, H, D, page, room, kind)


def test_tracking_arrays_of_any_alignment():
    """weights and pos one element past a multiple of 16 bytes, against aligned ones."""
    got = []
    for shift in (0, 1):
        torch.manual_seed(1)
        c = bcq.KVCache.new(2, 300, 2, 64, page_tokens=16)
        n = c.batch * c.heads * c.room
        w = torch.zeros(n + 1, device="cuda")[shift:n + shift].view(c._slots)
        pos = torch.zeros(n + 1, dtype=torch.int32, device="cuda")[shift:n + shift].view(c._slots)
        c.lens.copy_(torch.tensor([280, 140]))
        x = torch.randn((2, 2, 280, 2, 64), dtype=torch.float16, device="cuda")
        q = torch.randn((2, 4, 6, 64), dtype=torch.float16, device="cuda")
        o = torch.empty_like(q)
        bcq.bcq_kv_append(c, x[0], x[1], weights=w, pos=pos)
        bcq.bcq_kv_attend(c, q, o, weights=w)
        bcq.bcq_kv_evict(c, 131, 11, w, pos)
        got.append((o, w[..., :131].clone(), pos[..., :131].clone(), c.lens, c.k_codes, c.v_codes,
                    c.scales))
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------ together


def test_decode_loop_captured():
    """Append, attend and evict of a decode loop as a graph, its lengths on the device, against
    the same calls made one by one."""
    B, H, G, D, keep = 3, 2, 4, 64, 40
    state = []
    for _ in range(2):
        c = bcq.KVCache.new(B, keep + 8, H, D, page_tokens=16)
        state.append((c,) + c.tracking())
    x = torch.empty((2, B, 1, H, D), dtype=torch.float16, device="cuda")
    q = torch.empty((B, 1, H * G, D), dtype=torch.float16, device="cuda")
    positions = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    spaces = [(bcq.new_kv_workspace(s[0], 1, H * G, weights=True),
               bcq.new_kv_evict_workspace(s[0], keep)) for s in state]

    def step(k):
        c, w, pos = state[k]
        c.lens.add_(1)
        bcq.bcq_kv_append(c, x[0], x[1], positions=positions, weights=w, pos=pos)
        bcq.bcq_kv_attend(c, q, outs[k], weights=w, workspace=spaces[k][0])
        bcq.bcq_kv_evict(c, keep, 8, w, pos, workspace=spaces[k][1])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    torch.manual_seed(0)
    for i in range(60):
        x.normal_()
        q.normal_()
        positions.fill_(i)
        graph.replay()
        step(1)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]), i
        n = min(i + 1, keep)
        for a, b in zip(state[0][1:], state[1][1:]):
            assert torch.equal(a[..., :n], b[..., :n]), i
    assert state[0][0].lens.tolist() == [keep] * B
    pos = state[0][2][..., :keep]
    assert (pos.sort(-1).values[..., -8:] == torch.arange(52, 60, device="cuda")).all()


def test_on_another_stream():
    c = bcq.KVCache.new(2, 256, 2, 128)
    x = torch.randn((2, 2, 200, 2, 128), device="cuda")
    q = torch.randn((2, 1, 8, 128), device="cuda")
    o, want = torch.empty_like(q), torch.empty_like(q)
    c.lens.fill_(200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bcq.bcq_kv_append(c, x[0], x[1], stream=side)
    bcq.bcq_kv_attend(c, q, o, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    bcq.bcq_kv_attend(c, q, want)
    assert torch.equal(o, want)
