"""Refusals of the low-bit serving operators, without a GPU: every call here is rejected (or has
nothing to do) before any HIP call, so the addresses are never followed."""

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
    """The status of a call with some named arguments changed."""
    a = dict(args)
    assert set(change) <= set(a), change
    a.update(change)
    return getattr(lib, fn)(*a.values())


QUANTIZE = dict(X=A, dtype=F16, rows=3, K=100, ldx=104, codes=A, ldc=112, scales=A, stream=None)
GEMM = dict(A=A, a_scales=A, T=40, lda=112, W=A, w_scales=A, M=50, K=100, ldw=112, bias=None, Y=A,
            ldy=50, dtype=F16, workspace=A, bytes=1 << 30, stream=None)
LINEAR = dict(X=A, T=40, ldx=104, W=A, w_scales=A, M=50, K=100, ldw=112, bias=None, Y=A, ldy=50,
              dtype=F16, workspace=A, bytes=1 << 30, stream=None)

PRODUCT_BAD = [
    (dict(T=-1), INVALID), (dict(T=(1 << 20) + 1), INVALID), (dict(M=0), INVALID),
    (dict(M=1 << 24), INVALID), (dict(K=0), INVALID), (dict(K=131072, ldw=131072), INVALID),
    (dict(dtype=0), INVALID), (dict(dtype=3), INVALID), (dict(W=None), INVALID),
    (dict(w_scales=None), INVALID), (dict(Y=None), INVALID), (dict(ldw=96), INVALID),
    (dict(ldy=49), INVALID), (dict(W=A + 8), ALIGNMENT), (dict(ldw=120), ALIGNMENT),
    (dict(w_scales=A + 2), ALIGNMENT), (dict(Y=A + 1), ALIGNMENT), (dict(bias=A + 1), ALIGNMENT),
    (dict(workspace=None), INVALID), (dict(bytes=0), INVALID), (dict(workspace=A + 8), ALIGNMENT),
]


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 24), INVALID), (dict(K=0), INVALID),
    (dict(K=131072, ldx=131072, ldc=131072), INVALID), (dict(dtype=0), INVALID),
    (dict(X=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(ldx=96), INVALID), (dict(ldc=96), INVALID), (dict(X=A + 2), ALIGNMENT),
    (dict(ldx=101), ALIGNMENT), (dict(codes=A + 8), ALIGNMENT), (dict(ldc=120), ALIGNMENT),
    (dict(scales=A + 2), ALIGNMENT), (dict(rows=0, X=None, codes=None, scales=None), OK),
])
def test_quantize(lib, change, want):
    assert call(lib, "bcq_int_quantize", QUANTIZE, **change) == want


@pytest.mark.parametrize("change,want", PRODUCT_BAD + [
    (dict(A=None), INVALID), (dict(a_scales=None), INVALID), (dict(lda=96), INVALID),
    (dict(A=A + 8), ALIGNMENT), (dict(lda=120), ALIGNMENT), (dict(a_scales=A + 2), ALIGNMENT),
    (dict(T=0, A=None, a_scales=None, Y=None, workspace=None, bytes=0), OK),
])
def test_gemm(lib, change, want):
    assert call(lib, "bcq_int_gemm", GEMM, **change) == want


@pytest.mark.parametrize("change,want", PRODUCT_BAD + [
    (dict(X=None), INVALID), (dict(ldx=96), INVALID), (dict(X=A + 8), ALIGNMENT),
    (dict(ldx=100), ALIGNMENT), (dict(T=0, X=None, Y=None, workspace=None, bytes=0), OK),
])
def test_linear(lib, change, want):
    assert call(lib, "bcq_int_linear", LINEAR, **change) == want


def test_int_workspace(lib):
    size = lib.bcq_int_workspace_bytes
    need = size(40, 50, 100)
    assert need >= 40 * 112 + 40 * 4
    assert call(lib, "bcq_int_linear", LINEAR, bytes=need - 1) == INVALID
    assert call(lib, "bcq_int_gemm", GEMM, bytes=need - 1) == INVALID
    for bad in [(-1, 50, 100), (0, 50, 100), (40, 0, 100), (40, 50, 0), (40, 50, 131072)]:
        assert size(*bad) == 0
    # the largest call's sums are counted in 64 bits
    assert size(1 << 20, (1 << 24) - 1, 131071) > (1 << 20) * 131072


def cache(**change):
    a = dict(batch=2, heads=2, head_dim=128, page_tokens=64, num_pages=8, max_pages=4, k_codes=A,
             v_codes=A, scales=A, page_table=A, lens=A)
    assert set(change) <= set(a), change
    a.update(change)
    return ctypes.byref(lowbit._KVCache(*a.values()))


CACHE_BAD = [
    (dict(k_codes=None), INVALID), (dict(v_codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(page_table=None), INVALID), (dict(lens=None), INVALID), (dict(batch=0), INVALID),
    (dict(batch=(1 << 16) + 1), INVALID), (dict(heads=0), INVALID),
    (dict(heads=(1 << 12) + 1), INVALID), (dict(num_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 30), INVALID),
    (dict(batch=1 << 11, heads=1 << 11), INVALID),  # more rows than a launch has workgroups
    (dict(batch=1 << 10, heads=1 << 4, max_pages=1 << 14), INVALID),  # 2^34 cached vectors
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
    (dict(page_tokens=8), UNSUPPORTED), (dict(page_tokens=48), UNSUPPORTED),
    (dict(page_tokens=512), UNSUPPORTED), (dict(k_codes=A + 8), ALIGNMENT),
    (dict(v_codes=A + 8), ALIGNMENT), (dict(scales=A + 8), ALIGNMENT),
    (dict(page_table=A + 2), ALIGNMENT), (dict(lens=A + 2), ALIGNMENT),
]
VECTORS = dict(cache=cache(), n=3, K=A, kb=1, kt=1, kh=1, V=A, vb=1, vt=1, vh=1, dtype=F16)
APPEND = dict(VECTORS, positions=None, weights=None, pos=None, stream=None)
READ = dict(VECTORS, stream=None)
ATTEND = dict(cache=cache(), Q=A, n=3, heads=4, qb=1, qt=1, qh=1, O=A, ob=1, ot=1, oh=1, dtype=F16,
              scale=ctypes.c_float(0.1), weights=None, workspace=A, bytes=1 << 40, stream=None)
EVICT = dict(cache=cache(), keep=100, recent=10, weights=A, pos=A, lens_out=A, weights_out=A,
             pos_out=A, workspace=A, bytes=1 << 40, stream=None)
ENTRIES = {"bcq_kv_append": APPEND, "bcq_kv_read": READ, "bcq_kv_attend": ATTEND,
           "bcq_kv_evict": EVICT}


@pytest.mark.parametrize("fn", sorted(ENTRIES))
@pytest.mark.parametrize("change,want", CACHE_BAD)
def test_caches(lib, fn, change, want):
    assert call(lib, fn, ENTRIES[fn], cache=cache(**change)) == want


@pytest.mark.parametrize("fn", sorted(ENTRIES))
def test_no_cache(lib, fn):
    assert call(lib, fn, ENTRIES[fn], cache=None) == INVALID


@pytest.mark.parametrize("fn", ["bcq_kv_append", "bcq_kv_read"])
@pytest.mark.parametrize("change,want", [
    (dict(n=-1), INVALID), (dict(n=(1 << 24) + 1), INVALID), (dict(dtype=0), INVALID),
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(K=A + 1), ALIGNMENT),
    (dict(V=A + 2, dtype=F32), ALIGNMENT), (dict(n=0, K=None, V=None), OK),
    (dict(n=1 << 24, cache=cache(batch=64)), INVALID),  # more vectors than are counted
])
def test_vectors(lib, fn, change, want):
    assert call(lib, fn, ENTRIES[fn], **change) == want


@pytest.mark.parametrize("name", ["positions", "weights", "pos"])
def test_append_tracking_alignment(lib, name):
    assert call(lib, "bcq_kv_append", APPEND, **{name: A + 2}) == ALIGNMENT


@pytest.mark.parametrize("change,want", [
    (dict(n=-1), INVALID), (dict(n=(1 << 24) + 1), INVALID), (dict(heads=0), INVALID),
    (dict(heads=3), INVALID), (dict(heads=1 << 17), INVALID),
    (dict(n=1 << 24, heads=32), INVALID), (dict(dtype=0), INVALID),
    (dict(scale=ctypes.c_float(float("inf"))), INVALID),
    (dict(scale=ctypes.c_float(float("nan"))), INVALID), (dict(Q=None), INVALID),
    (dict(O=None), INVALID), (dict(Q=A + 1), ALIGNMENT), (dict(O=A + 2, dtype=F32), ALIGNMENT),
    (dict(weights=A + 2), ALIGNMENT), (dict(weights=A, workspace=None), INVALID),
    (dict(weights=A, bytes=15), INVALID), (dict(weights=A, workspace=A + 8), ALIGNMENT),
    (dict(n=0, Q=None, O=None, workspace=None, bytes=0), OK),
])
def test_attend(lib, change, want):
    assert call(lib, "bcq_kv_attend", ATTEND, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(keep=0, recent=0), INVALID), (dict(recent=-1), INVALID), (dict(recent=101), INVALID),
    (dict(weights=None), INVALID), (dict(pos=None), INVALID), (dict(lens_out=None), INVALID),
    (dict(weights_out=None), INVALID), (dict(pos_out=None), INVALID),
    (dict(weights=A + 2), ALIGNMENT), (dict(pos=A + 2), ALIGNMENT), (dict(lens_out=A + 2), ALIGNMENT),
    (dict(weights_out=A + 2), ALIGNMENT), (dict(pos_out=A + 2), ALIGNMENT),
    (dict(workspace=None), INVALID), (dict(bytes=0), INVALID), (dict(workspace=A + 8), ALIGNMENT),
])
def test_evict(lib, change, want):
    assert call(lib, "bcq_kv_evict", EVICT, **change) == want


def test_kv_workspaces(lib):
    size = lib.bcq_kv_workspace_bytes
    for c, _ in CACHE_BAD:
        assert size(cache(**c), 1, 4, 1) == 0
        assert lib.bcq_kv_evict_workspace_bytes(cache(**c), 16) == 0
    assert size(cache(), -1, 4, 1) == size(cache(), 0, 4, 1) == size(cache(), 1, 3, 1) == 0
    assert size(cache(), 1, 4, 1) > 0
    assert lib.bcq_kv_evict_workspace_bytes(cache(), 0) == 0
    need = lib.bcq_kv_evict_workspace_bytes(cache(), 100)
    assert call(lib, "bcq_kv_evict", EVICT, bytes=need - 1) == INVALID
    # counted in 64 bits
    wide = cache(batch=1 << 12, heads=8, page_tokens=256, max_pages=1 << 10)
    assert lib.bcq_kv_evict_workspace_bytes(wide, 1 << 17) > 1 << 34


def test_binding_refuses_host_tensors_and_other_shapes():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros((2, 32)), torch.zeros((4, 32), dtype=torch.int8)
    with pytest.raises(ValueError, match="device tensor"):
        bcq.bcq_int_quantize(x)
    with pytest.raises(ValueError, match="device tensor"):
        bcq.bcq_int_linear(x, w, torch.zeros(4), torch.zeros((2, 4)))
    with pytest.raises(ValueError, match="device tensor"):
        bcq.bcq_int_gemm(w, torch.zeros(4), w, torch.zeros(4), torch.zeros((4, 4)))
    with pytest.raises(ValueError, match="device tensor"):
        bcq.KVCache.new(1, 32, 1, 64, page_tokens=16, device="cpu")
    with pytest.raises(ValueError, match="2-D"):
        bcq.KVCache(x, x, x, x, x)
