"""bcq_kv_attend_packed on the GPU, held to what test_lowbit_accuracy says of attention over the
4-bit cache: sequences of unlike lengths and numbers of new tokens, with and without shared pages."""

import sys

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402
from test_gpu_kv import device  # noqa: E402
from test_lowbit_accuracy import definition, outputs_hold  # noqa: E402

DT = {"f16": (torch.float16, np.float16), "f32": (torch.float32, np.float32)}


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def packed_cache(lens, H, D, page, shared, seed, k_mean=1.0, width=None):
    """A host cache of random vectors whose sequences share their first pages; entries past the
    lengths name no page and unused slots hold NaN scales."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    width = width or max(shared, -(-max(max(lens), 1) // page)) + 1
    pages = shared + B * (width - shared)
    ids = rng.permutation(pages)
    table = np.concatenate([np.tile(ids[:shared], (B, 1)),
                            ids[shared:].reshape(B, width - shared)], axis=1)
    c = lb.Cache(pages, H, page, D, table, lens)
    c.k[:] = rng.integers(0, 256, c.k.shape)
    c.v[:] = rng.integers(0, 256, c.v.shape)
    c.s[:] = np.nan
    mean = rng.normal(size=(H, D)) * k_mean
    for b, L in enumerate(lens):
        for h in range(H):
            first = 0 if b == 0 else min(shared * page, L)
            last = max(L, shared * page) if b == 0 else L
            for t, (k, v) in enumerate(rng.normal(size=(max(last - first, 0), 2, D)), first):
                c.put(b, h, t, k + mean[h], v)
    for b in range(B):
        c.table[b, max(-(-max(int(lens[b]), 0) // page), shared):] = [-1, 1 << 30][b % 2]
    return c


def reference(c, q, starts, scale):
    """Outputs of packed queries [T][Hq][D], zeros for tokens of no sequence."""
    out = np.zeros(q.shape)
    for b in range(len(c.lens)):
        s, e = starts[b], starts[b + 1]
        if e > s:
            one = lb.Cache(1, c.H, c.page, c.D, c.table[b:b + 1], c.lens[b:b + 1])
            one.k, one.v, one.s = c.k, c.v, c.s
            out[s:e] = definition(one, q[None, s:e], scale)[0][0]
    return out


def attend(c, q, starts, shared, scale=None, max_n=None, dev=None, out=None, **kw):
    dev = dev or device(c)
    x = torch.from_numpy(q).cuda()
    o = torch.full_like(x, 7) if out is None else out
    n = int(np.diff(starts).max()) if max_n is None else max_n
    bcq.bcq_kv_attend_packed(dev, x, o, torch.from_numpy(np.asarray(starts, np.int32)).cuda(), n,
                             shared_pages=shared, scale=scale, **kw)
    return o.cpu().numpy()


def check(lens, news, Hq, H, D, page, shared, dtype, seed=0, first=0, spare=0, scale=None, **kw):
    c = packed_cache(lens, H, D, page, shared, seed + D, **kw)
    starts = np.concatenate([[0], np.cumsum(news)]) + first
    T = int(starts[-1]) + spare
    q = np.random.default_rng(seed + 1).normal(size=(T, Hq, D)).astype(DT[dtype][1])
    got = attend(c, q, starts, shared, scale)
    ref = reference(c, q, starts, float(np.float32(D ** -0.5 if scale is None else scale)))
    assert (got[:first] == 7).all() and (got[starts[-1]:] == 7).all()
    mine = slice(first, int(starts[-1]))
    assert np.isfinite(got[mine]).all()
    assert outputs_hold(got[mine], ref[mine])
    # each sequence by itself, as a small one is little of the whole
    for s, e in zip(starts[:-1], starts[1:]):
        if e > s:
            assert outputs_hold(got[s:e], ref[s:e]) or not ref[s:e].any()
            if not ref[s:e].any():
                assert not got[s:e].any()


# lens, new tokens, heads, cached heads, D, page, shared pages
WAYS = [
    ([1], [1], 1, 1, 64, 16, 0),
    ([700], [1], 8, 2, 128, 64, 0),  # split
    ([15, 16, 17, 0, 300], [1, 1, 1, 0, 1], 4, 2, 128, 16, 0),
    ([31, 200, 64], [1, 0, 2], 8, 1, 256, 32, 0),
    ([90, 33, 500], [5, 3, 8], 8, 2, 64, 16, 0),  # up to 32 rows
    ([90, 400, 33], [12, 16, 1], 8, 2, 128, 16, 0),  # two waves a sequence
    ([40, 300], [17, 8], 2, 1, 256, 16, 0),
    ([300, 90, 201], [130, 90, 1], 4, 2, 64, 64, 0),  # whole and partial prompts, a token
    ([150, 1, 129, 40], [150, 1, 129, 1], 7, 1, 128, 16, 0),
    ([600, 60], [70, 60], 4, 1, 128, 128, 0),  # many rows, split
    ([260], [40], 4, 2, 256, 64, 0),
    ([200, 70, 90], [1, 1, 1], 8, 2, 128, 16, 4),  # shared pages
    ([300, 290], [1, 1], 16, 2, 64, 16, 17),  # an odd number of them
    ([64, 65, 64, 100], [1, 1, 0, 3], 4, 2, 128, 64, 1),  # nothing behind them
    ([400, 390, 395], [20, 1, 5], 8, 2, 128, 16, 23),  # rows of 80, 4 and 20
    ([200, 180, 190, 170, 210, 205], [8] * 6, 8, 1, 256, 32, 5),  # 384 rows together
    ([200, 180, 190, 170, 210, 205], [5, 4, 3, 2, 1, 40], 8, 1, 64, 32, 5),
    ([500, 300], [150, 200], 2, 2, 64, 32, 6),  # many rows only: nothing is read together
]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,news,Hq,H,D,page,shared", WAYS)
def test_every_way(lens, news, Hq, H, D, page, shared, dtype):
    say("kv_attend_packed", lens, news, Hq, H, D, page, shared, dtype)
    check(lens, news, Hq, H, D, page, shared, dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_short_sequences_and_spare_rows(dtype):
    """More new tokens than the sequence has, sequences shorter than the shared pages, none at all;
    rows before the first and behind the last are left as they were."""
    say("kv_attend_packed short", dtype)
    check([20, 3, 0, 33], [29, 9, 4, 1], 3, 1, 64, 16, 0, dtype, first=5, spare=7)
    check([20, 3, 0, 33, -5], [4, 9, 4, 1, 2], 3, 1, 64, 16, 2, dtype, spare=3)
    check([40, 3, 33], [40, 1, 2], 2, 2, 128, 16, 2, dtype, first=1)


@pytest.mark.parametrize("B,H,D", [(100, 1, 64), (300, 2, 64), (600, 1, 128)])
@pytest.mark.parametrize("shared", [0, 2])
def test_many_sequences(B, H, D, shared):
    say("kv_attend_packed of", B, H, D, shared)
    rng = np.random.default_rng(B)
    lens = shared * 16 + rng.integers(1, 30, B)
    news = np.minimum(lens - shared * 16, np.where(rng.random(B) < 0.05, 30, rng.integers(0, 3, B)))
    check([int(n) for n in lens], [int(n) for n in news], 4 * H, H, D, 16, shared, "f16", seed=B)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 3e7, -1e9, 1e31, 3.4e38])
def test_scores_of_any_size(scale, dtype):
    say("kv_attend_packed scale", scale, dtype)
    check([300, 150, 201], [1, 40, 1], 4, 2, 64, 16, 3, dtype, scale=scale)


def test_strides():
    """Queries as a slice of a projection, outputs as columns of a wider matrix, odd rows."""
    say("kv_attend_packed strides")
    lens, news, Hq, H, D = [70, 40, 33], [1, 20, 3], 4, 2, 64
    c = packed_cache(lens, H, D, 16, 0, 1)
    dev = device(c)
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(starts[-1])
    for pad in (0, 1, 8):
        q = np.random.default_rng(2).normal(size=(T, 3 * Hq, D + pad)).astype(np.float16)
        x = torch.from_numpy(q).cuda()[:, Hq:2 * Hq, pad:]
        whole = torch.full((T, Hq, 2 * D + pad), 7.0, dtype=torch.float16, device="cuda")
        o = whole[:, :, D:2 * D]
        bcq.bcq_kv_attend_packed(dev, x, o, torch.from_numpy(starts).cuda(), 20)
        ref = reference(c, q[:, Hq:2 * Hq, pad:], starts, float(np.float32(D ** -0.5)))
        assert outputs_hold(o.cpu().numpy(), ref)
        assert (whole[:, :, :D] == 7).all() and (whole[:, :, 2 * D:] == 7).all()


def test_as_kv_attend():
    """Equal numbers of tokens: as near to bcq_kv_attend as fp32 roundings let two orders be."""
    say("kv_attend_packed and kv_attend")
    lens, n, Hq, H, D = [500, 130, 300], 3, 8, 2, 128
    c = packed_cache(lens, H, D, 64, 0, 5)
    dev = device(c)
    q = torch.randn((3, n, Hq, D), device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    bcq.bcq_kv_attend(dev, q, a)
    bcq.bcq_kv_attend_packed(dev, q.view(3 * n, Hq, D), b.view(3 * n, Hq, D),
                             torch.arange(0, 10, 3, dtype=torch.int32, device="cuda"), n)
    assert (a - b).norm() <= 4e-6 * a.norm()


def test_starts_that_are_none():
    """Starts that fall, pass T or are negative, and a max_n that is too small: nothing outside the
    arrays is read or written (outputs are of no meaning)."""
    say("kv_attend_packed odd starts")
    c = packed_cache([70, 40, 33, 90], 2, 64, 16, 1, 1)
    dev = device(c)
    T, Hq = 24, 4
    whole = torch.full((T + 16, Hq, 64), 7.0, device="cuda")
    q = torch.randn((T, Hq, 64), device="cuda")
    for starts in ([0, 24, 0, 24, 0], [24, 0, 24, 0, 24], [-9, 5, 1 << 30, 3, 24],
                   [0, 1, 2, 3, 1 << 30], [30, 40, 50, 60, 70]):
        for max_n in (1, 3, 24, 1 << 20):
            bcq.bcq_kv_attend_packed(dev, q, whole[8:8 + T],
                                     torch.tensor(starts, dtype=torch.int32, device="cuda"), max_n,
                                     shared_pages=1)
    torch.cuda.synchronize()
    assert (whole[:8] == 7).all() and (whole[8 + T:] == 7).all()


def test_entries_that_name_no_page():
    """A table of anything: reads stay in the cache, other sequences are as ever."""
    say("kv_attend_packed odd table")
    c = packed_cache([70, 40, 33], 2, 64, 16, 0, 1)
    q = np.random.default_rng(2).normal(size=(3, 4, 64)).astype(np.float32)
    want = attend(c, q, [0, 1, 2, 3], 0)
    c.table[1] = [-1, 1 << 30, -(1 << 31), 0, 7, 3][:c.table.shape[1]]
    got = attend(c, q, [0, 1, 2, 3], 0)
    assert (got[[0, 2]] == want[[0, 2]]).all()


def test_a_step_in_a_graph():
    """Captured once; replayed with other starts and lengths, between eager calls."""
    say("kv_attend_packed graph")
    c = packed_cache([300, 120, 90, 200], 2, 64, 16, 4, 3)
    dev = device(c)
    T, Hq = 40, 8
    q = np.random.default_rng(4).normal(size=(T, Hq, 64)).astype(np.float16)
    x = torch.from_numpy(q).cuda()
    o = torch.zeros_like(x)
    starts = torch.zeros(5, dtype=torch.int32, device="cuda")
    ws = bcq.new_kv_packed_workspace(dev, T, Hq, 30, shared_pages=4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bcq.bcq_kv_attend_packed(dev, x, o, starts, 30, shared_pages=4, workspace=ws)
    for new, lens in (([1, 1, 1, 1], [300, 120, 90, 200]), ([30, 1, 0, 2], [290, 100, 64, 199]),
                      ([2, 2, 30, 1], [101, 70, 84, 66]), ([1, 1, 1, 1], [300, 120, 90, 200])):
        s = np.concatenate([[0], np.cumsum(new)])
        starts.copy_(torch.from_numpy(s))
        dev.lens.copy_(torch.tensor(lens))
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        c.lens = np.array(lens, np.int32)
        got, ref = o.cpu().numpy(), reference(c, q, s, 0.125)
        assert outputs_hold(got[:s[-1]], ref[:s[-1]]) and (got[s[-1]:] == 7).all()
        eager = attend(c, q, s, 4, max_n=30, dev=dev)
        assert (eager == got).all()  # the same order of every sum


def test_not_finite_values():
    """NaN and infinities in the cache reach the rows that see them and no others; what lies behind
    a sequence's last token has no influence."""
    say("kv_attend_packed not finite")
    lens, news = [200, 90, 150], [1, 30, 2]
    for D, shared in ((64, 0), (128, 2), (256, 2)):
        c = packed_cache(lens, 1, D, 16, shared, 9)
        q = np.random.default_rng(2).normal(size=(33, 2, D)).astype(np.float32)
        starts = [0, 1, 31, 33]
        want = attend(c, q, starts, shared)
        for part in range(4):
            for value in (np.nan, np.inf):
                kept = c.s.copy()
                c.s[c.table[1, 75 // 16], 0, 75 % 16, part] = value  # its queries 15 on see it
                got = attend(c, q, starts, shared)
                same = [i for i in range(33) if not 16 <= i < 31]
                assert (got[same] == want[same]).all(), (D, part, value)
                assert not np.isfinite(got[16:31]).any() or (part < 2 and value == np.inf)
                c.s = kept


def test_more_rows_to_join_than_a_launch_has_room_for():
    """Past 2^22 rows the workgroups that join them take turns."""
    B, n, H, D, page = 4096, 8, 160, 64, 16
    say("kv_attend_packed joins", B * n * H, "rows")
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = bcq.KVCache.pool(B, 2 * page, B + 1, H, D, page)[0]
    cache.page_table[:, 0] = 0
    cache.page_table[:, 1] = torch.arange(1, B + 1, device="cuda")
    slots = torch.cat([torch.arange(page), torch.arange(B * n) // n * page + page
                       + torch.arange(B * n) % n]).cuda()
    for at in slots.split(4096):
        kv = torch.randn((2, len(at), H, D), generator=gen, device="cuda").half()
        bcq.bcq_kv_append_slots(cache, kv[0], kv[1], at)
    cache.lens[:] = page + n
    q = torch.randn((B * n, H, D), generator=gen, device="cuda").half()
    got, want = torch.full_like(q, 7), torch.empty_like(q)
    starts = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    bcq.bcq_kv_attend_packed(cache, q, got, starts, n, shared_pages=1)
    bcq.bcq_kv_attend(cache, q.view(B, n, H, D), want.view(B, n, H, D))
    # both round sums of 24 terms that agree to 1e-5 of the largest |v|, 4, once: half a
    # step each
    off = (got.float() - want.float()).abs()
    assert (off <= 2.0**-10 * want.float().abs() + 4e-5).all()
