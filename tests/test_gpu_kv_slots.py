"""Pages, slots and positions of a packed step (bcq_kv_reserve) and what is appended to and read
from those slots, on the GPU against their definitions, to the bit."""

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


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Server:
    """A cache's tables and its stack of free pages, on the host and on the device."""

    def __init__(self, lens, page, shared, pages, width, seed=0, H=1, D=64):
        rng = np.random.default_rng(seed)
        ids = rng.permutation(pages).astype(np.int32)
        self.page, self.shared = page, shared
        self.lens = np.array(lens, np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = shared
        for b, n in enumerate(lens):
            own = max(-(-n // page) - shared, 0)
            self.table[b, :shared] = ids[:shared]
            self.table[b, shared:shared + own] = ids[at:at + own]
            at += own
        assert at <= pages
        self.free = np.full(pages, -7, np.int32)
        self.count = pages - at
        self.free[:self.count] = ids[at:]
        z = lambda s, t: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        self.cache = bcq.KVCache(z((pages, H, page, D // 2), torch.uint8),
                                 z((pages, H, page // 4, 2 * D), torch.uint8),
                                 z((pages, H, page, 4), torch.float16), up(self.table),
                                 up(self.lens))
        self.dev = [up(self.free), up(np.array([self.count], np.int32))]

    def step(self, new, release, T, in_place=True, workspace=None):
        """One call, compared with the definition; the outputs (starts, slots, positions)."""
        B = len(self.lens)
        out = [torch.full(s, 99, dtype=t, device="cuda")
               for s, t in (((B + 1,), torch.int32), ((T,), torch.int64), ((T,), torch.int32))]
        kept = [torch.full_like(t, -9) for t in (self.cache.lens, self.cache.page_table,
                                                 *self.dev)]
        extra = {} if in_place else dict(zip(
            ("lens_out", "page_table_out", "free_pages_out", "free_count_out"), kept))
        bcq.bcq_kv_reserve(self.cache, up(np.array(new, np.int32)), *self.dev, *out,
                           release=None if release is None else up(np.array(release, np.int32)),
                           shared_pages=self.shared, workspace=workspace, **extra)
        torch.cuda.synchronize()
        lens, table, free, count, *packed = lb.reserve(
            self.lens, self.table, self.free, self.count, new, release, self.shared, self.page, T)
        got = (self.cache.lens, self.cache.page_table, *self.dev) if in_place else kept
        got = [t.cpu().numpy() for t in got]
        np.testing.assert_array_equal(got[0], lens)
        assert got[3][0] == count
        if in_place:
            np.testing.assert_array_equal(got[1], table)
            np.testing.assert_array_equal(got[2][:count], free[:count])
        else:
            pages = np.maximum(-(-lens // self.page), self.shared)[:, None]
            there = np.arange(table.shape[1]) < pages
            np.testing.assert_array_equal(got[1], np.where(there, table, -9))
            np.testing.assert_array_equal(got[2], np.where(np.arange(len(free)) < count, free, -9))
            for t, was in zip((self.cache.lens, self.cache.page_table, *self.dev),
                              (self.lens, self.table, self.free, [self.count])):
                np.testing.assert_array_equal(t.cpu().numpy(), was)
        for t, want in zip(out, packed):
            np.testing.assert_array_equal(t.cpu().numpy(), want)
        if in_place:
            self.lens, self.table, self.count = lens, table, count
            self.free = got[2]
        return out


# lens, new, release, shared, page, pages, width, T
STEPS = {
    "one token": ([0], [1], None, 0, 16, 3, 2, 1),
    "nothing asked": ([5, 0], [0, -3], [0, 0], 0, 16, 4, 2, 0),
    "the last place of a page": ([15, 16, 31], [1, 1, 1], None, 0, 16, 9, 3, 3),
    "ends and starts anew": ([40, 33, 0], [20, 1, 50], [1, 0, 1], 0, 16, 12, 4, 71),
    "gets its own pages back": ([64], [64], [1], 0, 16, 4, 4, 64),
    "too few pages for the second": ([0, 0, 15, 16], [16, 48, 1, 1], None, 0, 16, 5, 4, 80),
    "too few places": ([0, 0, 3], [10, 20, 4], None, 0, 32, 8, 2, 29),
    "past its table": ([30, 1], [3, 5], None, 0, 16, 6, 2, 8),
    "shared pages": ([32, 40, 0, 70], [1, 9, 5, 100], [0, 0, 0, 1], 2, 16, 20, 9, 200),
    "only shared pages": ([64, 64], [0, 0], [1, 0], 4, 16, 4, 4, 5),
    "room behind the last token": ([10], [5], None, 0, 256, 2, 1, 40),
}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("name", STEPS)
def test_step(name, in_place):
    say("kv_reserve", name, in_place)
    lens, new, release, shared, page, pages, width, T = STEPS[name]
    Server(lens, page, shared, pages, width).step(new, release, T, in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,page,shared,longest", [(70, 16, 0, 300), (1000, 64, 3, 90),
                                                   (1025, 16, 1, 40), (2500, 32, 0, 70)])
def test_a_server_at_work(B, page, shared, longest, in_place):
    """Steps of single tokens, prompts and requests that end, with more asked for than is there at
    times; no page belongs to two sequences or to one and the stack."""
    say("kv_reserve server", B, page, shared, longest, in_place)
    rng = np.random.default_rng(B)
    width = shared + -(-longest // page) + 1
    s = Server([shared * page] * B, page, shared, shared + B * (width - shared) * 2 // 5, width, B)
    ws = bcq.new_kv_reserve_workspace(s.cache)
    for _ in range(5):
        new = np.where(rng.random(B) < 0.2, rng.integers(0, longest, B), 1)
        release = (rng.random(B) < 0.25).astype(np.int32)
        s.step(new, release, int(new.sum() * rng.choice([0.7, 1, 1.2])), in_place, ws)
        if not in_place:
            s.step(new, release, int(new.sum()), True, ws)
        own = [s.table[b, shared:max(-(-n // page), shared)] for b, n in enumerate(s.lens)]
        used = np.concatenate(own + [s.free[:s.count], s.table[0, :shared]])
        assert len(used) == len(s.free) and len(set(used.tolist())) == len(used)


def test_entries_and_counts_that_name_no_page():
    """A stack and tables that hold anything: all that is written stays in its arrays."""
    say("kv_reserve odd state")
    s = Server([20, 33, 64, 0], 16, 0, 40, 4, 1)
    s.table[:] = [[-1, 1 << 30, -5, 7]] * 4
    s.cache.page_table.copy_(up(s.table))
    for count in (-3, 1 << 30, 39):
        s.count = min(max(count, 0), 40)
        s.free[:] = np.arange(40)
        s.dev[0].copy_(up(s.free))
        s.dev[1].fill_(count)
        s.lens = np.array([20, 33, 64, 0], np.int32)
        s.cache.lens.copy_(up(np.array([20, 33, 500, -4], np.int32)))
        s.step([5, 40, 3, 64], [1, 1, 1, 1], 200)
        s.table[:] = [[-1, 1 << 30, -5, 7]] * 4
        s.cache.page_table.copy_(up(s.table))


def test_a_step_in_a_graph():
    """Captured once, replayed with other requests each time, between eager calls."""
    say("kv_reserve graph")
    s = Server([3, 30, 16], 16, 0, 30, 6, 2)
    T = 40
    new, release = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    out = [torch.zeros(4, dtype=torch.int32, device="cuda"),
           torch.zeros(T, dtype=torch.int64, device="cuda"),
           torch.zeros(T, dtype=torch.int32, device="cuda")]
    ws = bcq.new_kv_reserve_workspace(s.cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bcq.bcq_kv_reserve(s.cache, new, *s.dev, *out, release=release, workspace=ws)
    for n, r in (([1, 1, 1], [0, 0, 0]), ([20, 1, 7], [1, 0, 0]), ([1, 0, 30], [0, 0, 1])):
        new.copy_(torch.tensor(n))
        release.copy_(torch.tensor(r))
        graph.replay()
        torch.cuda.synchronize()
        s.lens, s.table, free, s.count, *packed = lb.reserve(s.lens, s.table, s.free, s.count, n,
                                                             r, 0, 16, T)
        np.testing.assert_array_equal(s.cache.lens.cpu().numpy(), s.lens)
        np.testing.assert_array_equal(s.cache.page_table.cpu().numpy(), s.table)
        for t, want in zip(out, packed):
            np.testing.assert_array_equal(t.cpu().numpy(), want)
        s.free = s.dev[0].cpu().numpy()
        np.testing.assert_array_equal(s.free[:s.count], free[:s.count])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 16), (3, 8, 128, 64), (4, 2, 256, 16),
                                        (129, 5, 64, 32), (70, 3, 128, 256)])
@pytest.mark.parametrize("layout", ["whole", "projection", "odd"])
def test_append_and_read(T, H, D, page, dtype, layout):
    say("kv_append_slots", T, H, D, page, dtype, layout)
    tt, nt = DT[dtype]
    rng = np.random.default_rng(T + D)
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 2:
        slots[T // 2] = -1
        slots[T - 1] = pages * page + 5  # in no page
    x = rng.normal(size=(T, 4 * H, D)).astype(nt)
    x[0, H, :3] = [np.inf, 0, 1]
    if layout == "odd":  # rows that are not aligned to 4 channels
        whole = torch.zeros((T, 4 * H, D + 1), dtype=tt, device="cuda")
        whole[:, :, 1:] = up(x)
        dev = whole[:, :, 1:]
    else:
        dev = up(x)
    k, v = dev[:, H:2 * H], dev[:, 3 * H:]
    if layout == "whole":
        k, v = k.contiguous(), v.contiguous()
    host = lb.Cache(pages, H, page, D, [list(range(pages))], [0])
    host.k[:], host.v[:] = 17, 34
    host.s[:] = 2
    cache = bcq.KVCache(up(host.k), up(host.v), up(host.s), up(host.table), up(host.lens))
    bcq.bcq_kv_append_slots(cache, k, v, up(slots))
    ko, vo = (torch.full((T, H, D), 7.0, dtype=tt, device="cuda") for _ in range(2))
    bcq.bcq_kv_read_slots(cache, ko, vo, up(slots))
    torch.cuda.synchronize()
    there = (slots >= 0) & (slots < pages * page)
    for t in np.nonzero(there)[0]:
        for h in range(H):
            host.put(0, h, int(slots[t]), x[t, H + h], x[t, 3 * H + h])
    np.testing.assert_array_equal(cache.k_codes.cpu().numpy(), host.k)
    np.testing.assert_array_equal(cache.v_codes.cpu().numpy(), host.v)
    np.testing.assert_array_equal(cache.scales.cpu().numpy().view(np.uint16),
                                  host.s.view(np.uint16))
    for h in range(H):
        kk, vv, _ = host.get(0, h, np.where(there, slots, 0))
        for got, want in ((ko, kk), (vo, vv)):
            got = got[:, h].cpu().numpy()
            assert (got[~there] == 0).all()
            # zero + scale * code: the product is exact in fp32, the sum is rounded, then the type
            want = want.astype(np.float32).astype(nt)
            np.testing.assert_array_equal(got[there], want[there])


def test_the_same_as_append():
    """A step of equal numbers of tokens through slots, and through lengths."""
    say("kv_append_slots as kv_append")
    B, n, H, D, page = 3, 21, 4, 128, 16
    cache, free, count = bcq.KVCache.pool(B, 64, 12, H, D, page)
    other = bcq.KVCache.new(B, 64, H, D, page)
    k, v = torch.randn((2, B, n, H, D), device="cuda")
    T = B * n
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, slots = torch.empty(B + 1, **i32), torch.empty(T, dtype=torch.int64, device="cuda")
    positions = torch.empty(T, **i32)
    bcq.bcq_kv_reserve(cache, torch.full((B,), n, **i32), free, count, starts, slots, positions)
    bcq.bcq_kv_append_slots(cache, k.view(T, H, D), v.view(T, H, D), slots)
    other.lens.fill_(n)
    bcq.bcq_kv_append(other, k, v)
    outs = []
    for c in (cache, other):
        a, b = torch.empty_like(k), torch.empty_like(k)
        bcq.bcq_kv_read(c, a, b)
        outs += [a, b]
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert positions.view(B, n).tolist() == [list(range(n))] * B
    assert int(count) == 12 - B * 2


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_sign_of_a_zero(D):
    """A vector whose least element is a zero of either sign: four elements meet, then those of
    neighbours, pairs of them and so on, the later one winning among equals."""
    say("kv_append zeros", D)
    rng = np.random.default_rng(D)
    x = np.where(rng.random((40, 1, D)) < 0.5, 0.0, -0.0).astype(np.float32)
    x[::3] = np.where(rng.random(x[::3].shape) < 0.7, 1.5, x[::3])
    least = x[:, 0]
    pick = lambda a, b: np.where((a < b) | (a != a), a, b)  # noqa: E731
    for _ in range(2):
        least = pick(least[:, ::2], least[:, 1::2])
    at = np.arange(D // 4)
    for d in [1 << i for i in range(20) if 1 << i < D // 4]:
        least = pick(least, least[:, at ^ d])
    want = least[:, 0].astype(np.float16).view(np.uint16)
    k = up(x)
    cache = bcq.KVCache.new(1, 64, 1, D)
    cache.lens[:] = 40
    bcq.bcq_kv_append(cache, k.view(1, 40, 1, D), k.view(1, 40, 1, D))
    one = cache.scales.clone()
    cache.scales.fill_(7)
    bcq.bcq_kv_append_slots(cache, k, k, torch.arange(40, device="cuda"))
    for got in (one, cache.scales):
        got = got.cpu().numpy().view(np.uint16)[0, 0, :40]
        np.testing.assert_array_equal(got[:, 1], want)
        np.testing.assert_array_equal(got[:, 3], want)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,page,shared,longest", [(50, 16, 2, 700), (64, 64, 0, 2000),
                                                   (65, 16, 0, 3), (200, 16, 1, 3),
                                                   (256, 256, 1, 2), (257, 32, 0, 20)])
def test_a_server_of_any_size(B, page, shared, longest, in_place):
    test_a_server_at_work(B, page, shared, longest, in_place)


def test_more_tokens_than_a_grid_is_wide():
    """A grid's second dimension has 65535 workgroups at most, of four tokens of 256 channels."""
    T, D, page = 262150, 256, 256
    say("kv_append_slots", T, D)
    a, b = (bcq.KVCache.pool(1, T + page, T // page + 2, 1, D, page)[0] for _ in range(2))
    k, v = (torch.randn((T, 1, D), device="cuda").half() for _ in range(2))
    slots = torch.arange(T, device="cuda") + 3
    bcq.bcq_kv_append_slots(a, k, v, slots)
    for part in torch.arange(T, device="cuda").split(100000):
        bcq.bcq_kv_append_slots(b, k[part], v[part], slots[part])
    for x, y in ((a.k_codes, b.k_codes), (a.v_codes, b.v_codes), (a.scales, b.scales)):
        assert x.any() and torch.equal(x, y)
    got = torch.full((2, T, 1, D), 7.0, device="cuda", dtype=torch.float16)
    bcq.bcq_kv_read_slots(a, got[0], got[1], slots)
    for whole, x in zip(got, (k, v)):
        # half a step of 15, and the roundings of scale, zero and value
        step = (x.float().amax(2) - x.float().amin(2)) / 15
        assert ((whole.float() - x.float()).abs().amax(2) <= 0.5 * step + 0.02).all()
