"""The packed step's operators with work pending on other streams: each call with a workspace of
its own."""

import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def busy(product):
    """A few milliseconds of work on the current stream."""
    for _ in range(20):
        product @ product


def cache(lens, room, H=2, D=64):
    c = bcq.KVCache.new(len(lens), room, H, D)
    c.lens.fill_(room)
    kv = torch.randn((2, len(lens), room, H, D), device="cuda")
    bcq.bcq_kv_append(c, kv[0], kv[1])
    c.lens.copy_(torch.tensor(lens))
    return c


@pytest.mark.parametrize("B", [3, 70])
def test_attention_on_two_streams(B):
    """Up to 64 sequences and more; on the current stream and on another, the second queued while
    the first waits."""
    say("kv_attend_packed on two streams", B)
    lens = [600 - 5 * b for b in range(B)]
    new = [1 + 20 * (b == 1) for b in range(B)]
    c, T = cache(lens, 640), sum(new)
    starts = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    q = torch.randn((2, T, 4, 64), device="cuda")
    want, got = torch.empty_like(q), torch.empty_like(q)
    for i in (0, 1):
        bcq.bcq_kv_attend_packed(c, q[i], want[i], starts, 21)
    big = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        got.zero_()
        torch.cuda.synchronize()
        busy(big)
        bcq.bcq_kv_attend_packed(c, q[0], got[0], starts, 21)
        bcq.bcq_kv_attend_packed(c, q[1], got[1], starts, 21, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("B,T", [(40, 300), (40, 20000), (300, 9000)])
def test_reserve_on_two_streams(B, T):
    say("kv_reserve on two streams", B, T)
    g = torch.Generator(device="cuda").manual_seed(B)
    made, outs = [], []
    i32 = dict(dtype=torch.int32, device="cuda")
    for i in range(2):
        c, free, count = bcq.KVCache.pool(B, 600, B * 12, 1, 64, 64)
        new = torch.randint(0, 2 * T // B, (B,), generator=g, **i32)
        made.append((c, new, free, count))
        outs.append([torch.zeros(B + 1, **i32), torch.zeros(T, dtype=torch.int64, device="cuda"),
                     torch.zeros(T, **i32)])
    away = [[torch.zeros_like(t) for t in (c.lens, c.page_table, free, count)]
            for c, _, free, count in made]

    def call(i, stream=None):
        c, new, free, count = made[i]
        bcq.bcq_kv_reserve(c, new, free, count, *outs[i], lens_out=away[i][0],
                           page_table_out=away[i][1], free_pages_out=away[i][2],
                           free_count_out=away[i][3], stream=stream)

    call(0), call(1)
    want = [t.clone() for o in outs + away for t in o]
    big = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        for o in outs + away:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        busy(big)
        call(0)
        call(1, side)
        torch.cuda.synchronize()
        for t, w in zip((t for o in outs + away for t in o), want):
            assert torch.equal(t, w)


def test_norm_and_slots_on_a_given_stream():
    """What a call writes is ordered with its stream's work."""
    say("rms_norm and slots on another stream")
    side = torch.cuda.Stream()
    x = torch.randn((300, 512), device="cuda").half()
    gamma = torch.ones(512, device="cuda").half()
    big = torch.randn((4096, 4096), device="cuda")
    y, want = torch.empty_like(x), torch.empty_like(x)
    bcq.bcq_rms_norm(x, gamma, 1e-5, Y=want)
    c = bcq.KVCache.new(1, 304, 4, 128, 16)
    slots = torch.arange(300, device="cuda")
    k = torch.empty((300, 4, 128), device="cuda", dtype=torch.float16)
    ref = torch.empty_like(k)
    bcq.bcq_kv_append_slots(c, want.view(300, 4, 128), want.view(300, 4, 128), slots)
    bcq.bcq_kv_read_slots(c, ref, torch.empty_like(k), slots)
    c.scales.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy(big)
    bcq.bcq_rms_norm(x, gamma, 1e-5, Y=y, stream=side)
    bcq.bcq_kv_append_slots(c, y.view(300, 4, 128), y.view(300, 4, 128), slots, stream=side)
    bcq.bcq_kv_read_slots(c, k, torch.empty_like(k), slots, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(k, ref)
