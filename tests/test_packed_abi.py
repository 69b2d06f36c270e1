"""Refusals of the packed serving step's cache operators, without a GPU: every call here is
rejected (or has nothing to do) before any HIP call, so the addresses are never followed."""

import ctypes

import pytest

import binary_coded_precision_amd as bcq
from binary_coded_precision_amd import lowbit

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, -1, -2, -3
F16, F32 = 1, 2
A = 4096  # an aligned address


@pytest.fixture(scope="module")
def lib():
    return bcq.load()


def call(lib, fn, args, **change):
    a = dict(args)
    assert set(change) <= set(a), change
    a.update(change)
    return getattr(lib, fn)(*a.values())


def cache(**change):
    a = dict(batch=2, heads=2, head_dim=128, page_tokens=64, num_pages=8, max_pages=4, k_codes=A,
             v_codes=A, scales=A, page_table=A, lens=A)
    assert set(change) <= set(a), change
    a.update(change)
    return ctypes.byref(lowbit._KVCache(*a.values()))


SLOTS = dict(cache=cache(), T=3, slots=A, K=A, kt=1, kh=1, V=A, vt=1, vh=1, dtype=F16, stream=None)
RESERVE = dict(cache=cache(), new=A, release=A, shared=1, free=A, count=A, T=9, lens_out=A,
               table_out=A, free_out=A, count_out=A, starts=A, slots=A, positions=A, workspace=A,
               bytes=1 << 30, stream=None)
ENTRIES = {"bcq_kv_append_slots": SLOTS, "bcq_kv_read_slots": SLOTS, "bcq_kv_reserve": RESERVE}
CACHE_BAD = [
    (dict(k_codes=None), INVALID), (dict(lens=None), INVALID), (dict(batch=0), INVALID),
    (dict(heads=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_tokens=48), UNSUPPORTED),
    (dict(scales=A + 8), ALIGNMENT), (dict(page_table=A + 2), ALIGNMENT),
]


@pytest.mark.parametrize("fn", sorted(ENTRIES))
@pytest.mark.parametrize("change,want", CACHE_BAD)
def test_caches(lib, fn, change, want):
    assert call(lib, fn, ENTRIES[fn], cache=cache(**change)) == want


@pytest.mark.parametrize("fn", sorted(ENTRIES))
def test_no_cache(lib, fn):
    assert call(lib, fn, ENTRIES[fn], cache=None) == INVALID


@pytest.mark.parametrize("fn", ["bcq_kv_append_slots", "bcq_kv_read_slots"])
@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), INVALID), (dict(dtype=0), INVALID),
    (dict(dtype=3), INVALID), (dict(slots=None), INVALID), (dict(K=None), INVALID),
    (dict(V=None), INVALID), (dict(slots=A + 4), ALIGNMENT), (dict(K=A + 1), ALIGNMENT),
    (dict(V=A + 2, dtype=F32), ALIGNMENT), (dict(T=0, slots=None, K=None, V=None), OK),
    (dict(T=1 << 24, cache=cache(heads=16)), INVALID),  # more vectors than are counted
])
def test_slots(lib, fn, change, want):
    assert call(lib, fn, SLOTS, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), INVALID), (dict(shared=-1), INVALID),
    (dict(shared=5), INVALID), (dict(bytes=0), INVALID), (dict(workspace=A + 8), ALIGNMENT),
    (dict(slots=A + 4), ALIGNMENT),
] + [({name: None}, INVALID) for name in
     ("new", "free", "count", "lens_out", "table_out", "free_out", "count_out", "starts", "slots",
      "positions", "workspace")] + [({name: A + 2}, ALIGNMENT) for name in
     ("new", "release", "free", "count", "lens_out", "table_out", "free_out", "count_out",
      "starts", "positions")])
def test_reserve(lib, change, want):
    assert call(lib, "bcq_kv_reserve", RESERVE, **change) == want


def test_reserve_workspace(lib):
    size = lib.bcq_kv_reserve_workspace_bytes
    for c, _ in CACHE_BAD:
        assert size(cache(**c)) == 0
    need = size(cache())
    assert need >= 2 * (16 + 8) + 2 * 4 * 4
    assert call(lib, "bcq_kv_reserve", RESERVE, bytes=need - 1) == INVALID
    # counted in 64 bits
    assert size(cache(batch=1 << 16, heads=1, page_tokens=16, max_pages=1 << 13)) > 1 << 31
