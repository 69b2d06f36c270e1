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


ATTEND = dict(cache=cache(), Q=A, T=9, heads=4, qt=1, qh=1, starts=A, max_n=5, shared=1, O=A, ot=1,
              oh=1, dtype=F16, scale=ctypes.c_float(0.1), workspace=A, bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,want", CACHE_BAD + [(dict(batch=(1 << 12) + 1), INVALID)])
def test_attend_caches(lib, change, want):
    assert call(lib, "bcq_kv_attend_packed", ATTEND, cache=cache(**change)) == want
    assert lib.bcq_kv_packed_workspace_bytes(cache(**change), 9, 4, 5, 1) == 0


@pytest.mark.parametrize("change,want", [
    (dict(cache=None), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), INVALID),
    (dict(heads=0), INVALID), (dict(heads=3), INVALID), (dict(heads=1 << 17), INVALID),
    (dict(T=1 << 24, heads=32), INVALID), (dict(max_n=0), INVALID), (dict(max_n=-1), INVALID),
    (dict(shared=-1), INVALID), (dict(shared=5), INVALID), (dict(dtype=0), INVALID),
    (dict(dtype=3), INVALID), (dict(scale=ctypes.c_float(float("inf"))), INVALID),
    (dict(scale=ctypes.c_float(float("nan"))), INVALID), (dict(Q=None), INVALID),
    (dict(O=None), INVALID), (dict(starts=None), INVALID), (dict(Q=A + 1), ALIGNMENT),
    (dict(O=A + 2, dtype=F32), ALIGNMENT), (dict(starts=A + 2), ALIGNMENT),
    (dict(workspace=None), INVALID), (dict(bytes=15), INVALID), (dict(workspace=A + 8), ALIGNMENT),
    # more rows than a workspace counts
    (dict(T=1 << 22, heads=64, max_n=1 << 22,
          cache=cache(heads=1, page_tokens=256, max_pages=1 << 15)), INVALID),
    (dict(T=0, Q=None, starts=None, O=None, workspace=None, bytes=0), OK),
])
def test_attend(lib, change, want):
    assert call(lib, "bcq_kv_attend_packed", ATTEND, **change) == want


def test_attend_workspace(lib):
    size = lib.bcq_kv_packed_workspace_bytes
    assert size(cache(), 0, 4, 5, 1) == size(cache(), 9, 3, 5, 1) == size(cache(), 9, 4, 0, 0) == 0
    need = size(cache(), 9, 4, 5, 1)
    assert need > 0 and need == size(cache(), 9, 4, 5, 2)
    assert size(cache(), 9, 4, 1 << 30, 1) == size(cache(), 9, 4, 9, 1)  # at most T of one
    assert call(lib, "bcq_kv_attend_packed", ATTEND, bytes=need - 1) == INVALID
    # counted in 64 bits
    assert size(cache(page_tokens=256, max_pages=1 << 8), 1 << 20, 64, 1 << 20, 0) > 1 << 34
