"""The largest calls of append and read by slots that are refused, without a GPU: a launch has less
than 2^32 work items, each of which takes four channels of K and of V."""

import pytest

from test_packed_abi import INVALID, SLOTS, cache, call, lib  # noqa: F401


@pytest.mark.parametrize("fn", ["bcq_kv_append_slots", "bcq_kv_read_slots"])
@pytest.mark.parametrize("heads,dim,T", [(16, 64, 1 << 24), (8, 128, 1 << 24), (4, 256, 1 << 24),
                                         (1 << 12, 64, 63489), (1 << 12, 256, 15873)])
def test_more_work_items_than_a_launch_has(lib, fn, heads, dim, T):  # noqa: F811
    assert heads * (T * dim + (1 << 17)) >= 1 << 34
    assert call(lib, fn, SLOTS, T=T, cache=cache(heads=heads, head_dim=dim)) == INVALID
