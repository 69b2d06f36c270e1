"""Packed append and read of as many tokens as a call can have."""

import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def test_the_most_tokens_of_fifteen_heads():
    """2^24 tokens of 15 heads of 64 channels, 15/16 of the work items that a launch can have; the
    same vectors for each token, of which a few have slots."""
    T, H, D, page = 1 << 24, 15, 64, 64
    say("kv_append_slots", T, H, D)
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("takes 65 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = torch.randn((2, 1, H, D), generator=g, device="cuda").half()
    a, b = (bcq.KVCache.pool(1, 1024, 16, H, D, page)[0] for _ in range(2))
    at = torch.cat([torch.tensor([0, 15, 16, T // 2, T - 17, T - 16, T - 1]),
                    torch.randint(17, T - 17, (300,), generator=torch.Generator().manual_seed(2))])
    at = at.unique().cuda()
    few = torch.randperm(16 * page, generator=g, device="cuda")[:len(at)]
    slots = torch.full((T,), -1, device="cuda")
    slots[at] = few
    bcq.bcq_kv_append_slots(a, k.expand(T, H, D), v.expand(T, H, D), slots)
    n = len(at)
    bcq.bcq_kv_append_slots(b, k.expand(n, H, D), v.expand(n, H, D), few)
    for x, y in ((a.k_codes, b.k_codes), (a.v_codes, b.v_codes), (a.scales, b.scales)):
        assert x.any() and torch.equal(x, y)
    got = torch.full((2, T, H, D), 7.0, device="cuda", dtype=torch.float16)
    want = torch.empty((2, n, H, D), device="cuda", dtype=torch.float16)
    bcq.bcq_kv_read_slots(a, got[0], got[1], slots)
    bcq.bcq_kv_read_slots(b, want[0], want[1], few)
    for whole, x in zip(got, want):
        assert torch.equal(whole[at], x)
        whole[at] = 0
        assert not any(part.any() for part in whole.split(1 << 20))
    del got, whole
    torch.cuda.empty_cache()
