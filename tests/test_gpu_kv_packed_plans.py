"""How bcq_kv_attend_packed cuts large calls into items, against the definition in 64 bits: shared
pages in whole turns of the compute units, shares that are cut because a wave sums no more steps in
one go, tables with room past 2^16 tokens, and splits among more than 64 sequences."""

import sys

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402
from test_lowbit_accuracy import F16, FP32, definition, norm  # noqa: E402

DT = {"f16": torch.float16, "f32": torch.float32}


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def random_cache(lens, H, D, page, shared, seed):
    """Random codes and scales in scattered pages, the first `shared` the same for all; what no
    sequence has cached holds NaN scales and entries past the lengths name no page."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, lens = len(lens), torch.tensor(lens)
    width = max(shared, -(-int(lens.max()) // page)) + 1
    pages = shared + B * (width - shared)
    ids = torch.randperm(pages, generator=g, device="cuda").int().cpu()
    table = torch.cat([ids[:shared].expand(B, shared), ids[shared:].view(B, width - shared)], 1)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda",  # noqa: E731
                                    dtype=torch.uint8)
    # 15 steps of 0.2 to 0.3 about zero
    f = torch.rand((pages, H, page, 4), generator=g, device="cuda")
    f[..., 0::2] = 0.2 + 0.1 * f[..., 0::2]
    f[..., 1::2] = -1.9 + 0.3 * f[..., 1::2]
    slot = torch.arange(width * page)
    there = torch.zeros(pages * page, dtype=torch.bool)
    for b in range(B):
        at = slot[:lens[b]]
        there[table[b, at // page].long() * page + at % page] = True
        table[b, max(-(-int(lens[b]) // page), shared):] = [-1, 1 << 30][b % 2]
    f.masked_fill_(~there.view(pages, 1, page, 1).cuda(), float("nan"))
    return bcq.KVCache(byte(pages, H, page, D // 2), byte(pages, H, page // 4, 2 * D), f.half(),
                       table.contiguous().cuda(), lens.int().cuda())


def vectors(c, b, h, L):
    """Keys and values of one sequence's first L tokens, in 64 bits."""
    slot = torch.arange(L, device="cuda")
    page, line = c.page_table[b].long()[slot // c.page_tokens], slot % c.page_tokens
    d = torch.arange(c.head_dim, device="cuda")
    m = c.scales[page, h, line].double()
    k = c.k_codes[page, h, line][:, d // 2] >> (d % 2 * 4).to(torch.uint8) & 15
    byte, shift = (torch.from_numpy(x).cuda() for x in lb.v_place(c.head_dim))
    v = c.v_codes[page, h, line // 4].gather(1, byte + (line % 4 * 2)[:, None])
    v = v >> shift.to(torch.uint8) & 15
    return m[:, 1:2] + m[:, 0:1] * k, m[:, 3:4] + m[:, 2:3] * v


def reference(c, q, starts, scale):
    """The definition for packed queries [T][Hq][D], in 64 bits."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    G = q.shape[1] // c.heads
    for b, L in enumerate(c.lens.tolist()):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        last = L - n + torch.arange(n, device="cuda").repeat_interleave(G)
        hidden = torch.arange(L, device="cuda") > last[:, None]
        for h in range(c.heads):
            k, v = vectors(c, b, h, L)
            k = k.T.contiguous()
            x = q[starts[b]:starts[b + 1], h * G:(h + 1) * G].double().reshape(n * G, -1)
            for rows in torch.arange(n * G, device="cuda").split(max(1, (1 << 28) // L)):
                z = (x[rows] @ k).mul_(scale).masked_fill_(hidden[rows], -float("inf"))
                p = z.sub_(z.amax(1, keepdim=True)).exp_()
                i, g = rows // G, rows % G
                out[starts[b] + i, h * G + g] = (p @ v) / p.sum(1, keepdim=True)
    return out


def test_the_reference_is_the_definition():
    """On the device and from the oracle's bytes, where that can be looked at row by row."""
    say("kv_attend_packed plans: reference")
    for D, Hq, H in ((64, 4, 2), (128, 3, 1), (256, 2, 2)):
        c = random_cache([70, 41, 50], H, D, 16, 2, D)
        starts = [0, 3, 3, 12]
        q = torch.randn((12, Hq, D), device="cuda")
        got = reference(c, q, starts, D ** -0.5).cpu().numpy()
        host = lb.Cache(c.num_pages, H, 16, D, c.page_table.cpu().numpy(), c.lens.cpu().numpy())
        host.k, host.v, host.s = (t.cpu().numpy() for t in (c.k_codes, c.v_codes, c.scales))
        for b in range(3):
            one = lb.Cache(1, H, 16, D, host.table[b:b + 1], host.lens[b:b + 1])
            one.k, one.v, one.s = host.k, host.v, host.s
            mine = slice(starts[b], starts[b + 1])
            if starts[b + 1] > starts[b]:
                want = definition(one, q[None, mine].cpu().numpy(), D ** -0.5)[0][0]
                assert np.abs(got[mine] - want).max() < 1e-12


def check(lens, news, Hq, H, D, page, shared, dtype, seed=0, sums=0):
    """sums: additions that a lane makes in a row's longest sum.  Each is off by half a step, 2^-24
    of the sum so far, either way, so that N of them are off by about sqrt(N) of that at most, in
    the sum of the probabilities and in that of what they weigh."""
    say("kv_attend_packed plan", len(lens), lens[:2], max(news), Hq, H, D, page, shared, dtype)
    c = random_cache(lens, H, D, page, shared, seed + D)
    starts = [0] + np.cumsum(news).tolist()
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn((starts[-1], Hq, D), generator=g, device="cuda").to(DT[dtype])
    got = torch.full_like(q, 7)
    bcq.bcq_kv_attend_packed(c, q, got, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                             max(news), shared_pages=shared)
    ref = reference(c, q, starts, float(np.float32(D ** -0.5)))
    near = FP32 + 2 * sums**0.5 * 2.0**-24
    for s, e in [(0, starts[-1])] + list(zip(starts[:-1], starts[1:])):
        if e > s:
            out, want = got[s:e].cpu().numpy(), ref[s:e].cpu().numpy()
            own = 0 if dtype == "f32" else F16 * norm(want.astype(np.float16) - want)
            assert norm(out - want) <= own + near * norm(want), (s, e)


def grow(first, by, B):
    return [first + by * b for b in range(B)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,news,Hq,H,D", [
    (grow(8200, 7, 32), [1] * 32, 64, 8, 64),  # 17 shares of two blocks become 16
    (grow(8200, 7, 20), [1, 2] * 10, 64, 32, 64),  # 12 of one become 8
    (grow(8200, 7, 32), [1] * 32, 64, 8, 256),  # 12 of four become 8
    (grow(8100, 7, 100), [1] * 100, 64, 8, 128),  # 7 of seven become 4
])
def test_whole_turns(lens, news, Hq, H, D, dtype):
    """Shared pages of 8000 tokens whose items pass the compute units' number, which more shares of
    unlike lengths would leave idle for most of a turn."""
    check(lens, news, Hq, H, D, 64, 125, dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,news,Hq,H,shared", [
    ([70000], [1024], 64, 1, 0),  # a prompt's rows, one share by what there is to do
    ([70000] + [500] * 69, [1024] + [1] * 69, 64, 1, 0),
    (grow(70500, 1, 64), [1] * 64, 576, 9, 274),  # shared pages, one share by whole turns
    (grow(70500, 1, 75), [1] * 75, 512, 8, 274),
])
def test_shares_cut_by_length(lens, news, Hq, H, shared, dtype):
    """More than 2048 steps of 32 tokens where the card is full without another share, in tables
    with room past 2^16 tokens; a step adds eight terms to a lane's sums."""
    check(lens, news, Hq, H, 64, 256, shared, dtype, sums=8 * 2048)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n", [1, 20])
def test_a_sequence_past_two_to_the_eighteen(n, dtype):
    """One sequence in as many shares as a row can have."""
    check([300000], [n], 8, 1, 64, 256, 0, dtype, sums=8 * 147)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,news,Hq,H,D,page,shared", [
    # a prompt in 5 shares, single tokens in 2 or, behind shared pages of 3, in 1
    (grow(1000, 3, 80), [1] * 79 + [400], 8, 2, 64, 16, 0),
    (grow(1000, 3, 80), [1] * 79 + [400], 8, 2, 64, 16, 40),
    (grow(1000, 3, 300), [1] * 150 + [300] + [1] * 149, 8, 2, 128, 16, 20),  # in 4
    # prompts in 5 and 6 shares, drafted tokens in 2 and 3, sequences without tokens
    (grow(1000, 3, 66), [5] * 33 + [300] + [0] * 31 + [90], 4, 1, 256, 32, 10),
    (grow(1000, 3, 66), [5] * 33 + [300] + [0] * 31 + [90], 4, 1, 256, 32, 0),
])
def test_splits_among_many_sequences(lens, news, Hq, H, D, page, shared, dtype):
    check(lens, news, Hq, H, D, page, shared, dtype)
