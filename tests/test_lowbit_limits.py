"""The limits that bcq.h gives for the 4-bit cache's calls, from both sides, without a GPU: what is
within them is refused for the next reason (an address that is not aligned), before any HIP call."""

import pytest

import binary_coded_precision_amd as bcq
from test_lowbit_abi import A, ALIGNMENT, ATTEND, INVALID, VECTORS, cache, call

MOST = bcq.BCQ_KV_MAX_TOKENS


@pytest.fixture(scope="module")
def lib():
    return bcq.load()


@pytest.mark.parametrize("fn", ["bcq_kv_append", "bcq_kv_read"])
@pytest.mark.parametrize("n,shape,want", [
    (MOST, dict(batch=1, heads=1, head_dim=64), ALIGNMENT),
    (MOST + 1, dict(batch=1, heads=1, head_dim=64), INVALID),
    # 512 (n + 6) against 2^33 - 512
    (MOST - 8, dict(batch=8, heads=1, head_dim=64), ALIGNMENT),
    (MOST - 7, dict(batch=8, heads=1, head_dim=64), INVALID),
    (MOST // 4 - 8, dict(batch=2, heads=4, head_dim=256), ALIGNMENT),
    (MOST // 4 - 6, dict(batch=2, heads=4, head_dim=256), INVALID),
])
def test_new_tokens(lib, fn, n, shape, want):
    a = dict(VECTORS, cache=cache(**shape), n=n, K=A + 1)
    if fn == "bcq_kv_append":
        a.update(positions=None, weights=None, pos=None)
    assert call(lib, fn, dict(a, stream=None)) == want


@pytest.mark.parametrize("n,q_heads,batch,want", [
    (MOST, 16, 1, ALIGNMENT), (MOST + 1, 1, 1, INVALID), (1, 1 << 16, 1, ALIGNMENT),
    (1, (1 << 16) + 1, 1, INVALID),
    (MOST, 17, 1, INVALID), (1 << 12, 1 << 16, 1, ALIGNMENT), ((1 << 12) + 1, 1 << 16, 1, INVALID),
    (MOST, 16, 2, ALIGNMENT), (MOST, 16, 3, INVALID), (MOST // 2, 16, 4, ALIGNMENT),
    (MOST // 2 + 1, 16, 4, INVALID),
])
def test_queries(lib, n, q_heads, batch, want):
    a = dict(ATTEND, cache=cache(batch=batch, heads=1), n=n, heads=q_heads, Q=A + 1)
    assert call(lib, "bcq_kv_attend", a) == want
    bytes_ = lib.bcq_kv_workspace_bytes(cache(batch=batch, heads=1), n, q_heads, 1)
    assert (bytes_ > 0) == (want == ALIGNMENT)


def test_long_sequences_are_shared_out(lib):
    """No wave sums more than 2^16 tokens in one go, whatever the number of rows, up to what a
    launch can join; the workspace holds the parts."""
    def size(room, n, heads=1, q_heads=16, batch=1):
        c = cache(batch=batch, heads=heads, max_pages=room // 64)
        return lib.bcq_kv_workspace_bytes(c, n, q_heads, 0)

    part = 8 + 128 * 4  # of a row: a reference, a sum, outputs
    for n in (1 << 13, 1 << 20):  # enough workgroups without
        assert size(1 << 16, n) == 0
        for room, splits in ((1 << 17, 2), (3 << 16, 3), (1 << 22, 64), (1 << 24, 64)):
            assert splits * n * 16 * part <= size(room, n) < splits * n * 16 * part + 512
    # a decode step's four waves share a workgroup's tokens
    assert size(1 << 18, 1, heads=1 << 10, q_heads=1 << 10, batch=16) == 0
    got = size(1 << 19, 1, heads=1 << 10, q_heads=1 << 10, batch=8)
    assert 2 * (1 << 13) * part <= got < 2 * (1 << 13) * part + 512
    # more rows than a launch joins
    assert size(1 << 18, 1 << 24) == 0
