"""Binding of the low-bit serving operators: the 8-bit integer linear layer, the norm before it
and the 4-bit key/value cache (reserve, append, read, attend, evict).  Names and semantics are
those of ``include/bcq.h``; the package exports everything here.

The tensors of a call, and its ``stream`` if one is given, belong to one device, which need not be
the current one.
"""

from __future__ import annotations

import ctypes

BCQ_KV_MAX_TOKENS = 1 << 24
BCQ_KV_PACKED_MAX_BATCH = 1 << 12

_vp, _i32, _i64, _sz, _int = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                              ctypes.c_int)


class _KVCache(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("batch", "heads", "head_dim", "page_tokens", "num_pages",
                                    "max_pages")] + [
        (n, _vp) for n in ("k_codes", "v_codes", "scales", "page_table", "lens")]


_kc = ctypes.POINTER(_KVCache)
_strides = [_i64, _i64, _i64]

SIGNATURES = {
    "bcq_int_quantize": (_int, [_vp, _int, _i32, _i32, _i32, _vp, _i32, _vp, _vp]),
    "bcq_int_gemm": (_int, [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _i32,
                            _int, _vp, _sz, _vp]),
    "bcq_int_linear": (_int, [_vp, _i32, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _i32, _int,
                              _vp, _sz, _vp]),
    "bcq_int_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "bcq_rms_norm": (_int, [_vp, _i32, _vp, _i32, _vp, ctypes.c_double, _i32, _i32, _int, _vp,
                            _i32, _vp, _i32, _vp, _i32, _vp, _vp]),
    "bcq_kv_append": (_int, [_kc, _i32, _vp, *_strides, _vp, *_strides, _int, _vp, _vp, _vp,
                             _vp]),
    "bcq_kv_read": (_int, [_kc, _i32, _vp, *_strides, _vp, *_strides, _int, _vp]),
    "bcq_kv_reserve": (_int, [_kc, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                              _vp, _vp, _sz, _vp]),
    "bcq_kv_reserve_workspace_bytes": (_sz, [_kc]),
    "bcq_kv_append_slots": (_int, [_kc, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _int, _vp]),
    "bcq_kv_read_slots": (_int, [_kc, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _int, _vp]),
    "bcq_kv_attend": (_int, [_kc, _vp, _i32, _i32, *_strides, _vp, *_strides, _int,
                             ctypes.c_float, _vp, _vp, _sz, _vp]),
    "bcq_kv_workspace_bytes": (_sz, [_kc, _i32, _i32, _i32]),
    "bcq_kv_attend_packed": (_int, [_kc, _vp, _i32, _i32, _i64, _i64, _vp, _i32, _i32, _vp, _i64,
                                    _i64, _int, ctypes.c_float, _vp, _sz, _vp]),
    "bcq_kv_packed_workspace_bytes": (_sz, [_kc, _i32, _i32, _i32, _i32]),
    "bcq_kv_evict": (_int, [_kc, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bcq_kv_evict_workspace_bytes": (_sz, [_kc, _i32]),
}
EXPORTS = tuple(SIGNATURES)


# The loaded library and torch, bound at the first call: these operators are called once a layer
# and token, so a call does no more than read its tensors' descriptions and pass them on.
_lib = None
torch = None


def _bind():
    global _lib, torch
    import torch as _torch

    import binary_coded_precision_amd as pkg

    torch = _torch
    _lib = pkg.load()
    return _lib


def _fail(fn: str, status: int):
    import binary_coded_precision_amd as pkg

    raise pkg.BCQError(fn, status)


def _pad16(n: int) -> int:
    return (n + 15) // 16 * 16


def _device(name: str, t) -> int:
    """The device of a call, that of its tensor t."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.get_device()


def _raw(dev: int, stream) -> int:
    """The raw stream a call goes to: the given one, or the current one of its device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("stream must belong to device %d, as the call's tensors do" % dev)
    return stream.cuda_stream


def _there(dev: int, call, *args):
    """A call made again with its tensors' device current: launches go to that one."""
    with torch.cuda.device(dev):
        return call(*args)


def _empty(shape, dtype, device, stream):
    """A tensor that a call on `stream` (None: the current one) may write at once: memory of that
    stream's, as another's may still be in use there by what was queued before it was freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(n_bytes: int, device, stream):
    """A workspace of n_bytes for a call on `stream`."""
    return _empty(max(n_bytes, 1), torch.uint8, device, stream)


def _space(t, dev: int):
    """(address, bytes) of a workspace."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor on the call's device")
    return t.data_ptr(), t.nbytes


def _float(name: str, t, dev: int) -> int:
    """The dtype code of a tensor of fp16 or fp32 on the call's device."""
    if t.get_device() != dev:
        raise ValueError("%s must be a device tensor on the call's device" % name)
    d = t.dtype
    if d is torch.float16:
        return 1
    if d is torch.float32:
        return 2
    raise TypeError("%s must be float16 or float32, got %s" % (name, d))


def _plain(name: str, t, dtype, shape, dev: int) -> int:
    """The address of a contiguous tensor of this dtype and shape on the call's device."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s device tensor of shape %s on device %d, got "
                         "%s of %s on %s" % (name, dtype, tuple(shape), dev, tuple(t.shape),
                                             t.dtype, t.device))
    return t.data_ptr()


def _rows(name: str, t, rows: int, cols: int, read: int) -> int:
    """The leading dimension of a [rows][cols] matrix with unit inner stride whose every row
    can be read up to column `read`."""
    if t.shape != (rows, cols):
        raise ValueError("%s must be %d x %d, got %s" % (name, rows, cols, tuple(t.shape)))
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError("%s must have unit inner stride" % name)
    if rows < 2 and ld < read:
        ld = read
    if read > cols and rows:
        room = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
        if (rows - 1) * ld + read > room:
            raise ValueError("%s: the last row must be readable up to column %d" % (name, read))
    return ld


def _like(name: str, t, shape, dtype, dev: int):
    """(address, leading dimension) of a matrix of this shape [T][K] and dtype with unit inner
    stride on the call's device."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise ValueError("%s must be a %s device tensor of shape %s on device %d, got %s of %s on %s"
                         % (name, dtype, tuple(shape), dev, tuple(t.shape), t.dtype, t.device))
    ld, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ValueError("%s must have unit inner stride" % name)
    # a single row has no next one to be aligned with
    return t.data_ptr(), ld if shape[0] > 1 else _pad16(shape[1])


# ----------------------------------------------------------------------------- 8-bit products


def bcq_int_workspace_bytes(T: int, M: int, K: int) -> int:
    return int((_lib or _bind()).bcq_int_workspace_bytes(T, M, K))


def new_int_workspace(T: int, M: int, K: int, device="cuda"):
    """A device workspace for :func:`bcq_int_linear` and :func:`bcq_int_gemm`; calls that may
    overlap need separate ones."""
    return _workspace(bcq_int_workspace_bytes(T, M, K), device, None)


def bcq_int_quantize(X, codes=None, scales=None, stream=None):
    """Rounds each row of ``X`` [rows][K] (fp16 or fp32, rows 16-byte aligned) to 8 bits.

    Returns ``(codes, scales)``: int8 [rows][K] (a view of rows padded to 16 bytes with zeros)
    and fp32 [rows], allocated on ``stream`` unless given."""
    lib = _lib or _bind()
    dev = _device("X", X)
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_int_quantize, X, codes, scales, stream)
    raw = _raw(dev, stream)
    dt = _float("X", X, dev)
    rows, K = X.shape
    ldx = _rows("X", X, rows, K, K)
    if codes is None:
        codes = _empty((rows, _pad16(K)), torch.int8, X.device, stream)[:, :K]
    if scales is None:
        scales = _empty(rows, torch.float32, X.device, stream)
    if codes.dtype is not torch.int8 or codes.get_device() != dev:
        raise ValueError("codes must be an int8 device tensor on X's device")
    if rows == 1:
        ldx = _pad16(ldx)  # a single row has no next one to be aligned with
    r = lib.bcq_int_quantize(X.data_ptr(), dt, rows, K, ldx, codes.data_ptr(),
                             _rows("codes", codes, rows, K, _pad16(K)),
                             _plain("scales", scales, torch.float32, (rows,), dev), raw)
    if r:
        _fail("bcq_int_quantize", r)
    return codes, scales


def _product(W, w_scales, Y, T: int, bias, dev: int):
    """Checks what the two products share; (M, K, ldw, ldy, dtype, scales', bias' address)."""
    if W.dtype is not torch.int8:
        raise ValueError("W must be an int8 device tensor")
    M, K = W.shape
    return (M, K, _rows("W", W, M, K, _pad16(K)), _rows("Y", Y, T, M, M), _float("Y", Y, dev),
            _plain("w_scales", w_scales, torch.float32, (M,), dev),
            0 if bias is None else _plain("bias", bias, Y.dtype, (M,), dev))


def bcq_int_gemm(A, a_scales, W, w_scales, Y, bias=None, workspace=None, stream=None) -> None:
    """``Y[t][m] = (A[t] . W[m]) * (a_scales[t] * w_scales[m]) + bias[m]`` from 8-bit codes as
    :func:`bcq_int_quantize` returns them.  ``workspace`` as in :func:`bcq_int_linear`."""
    lib = _lib or _bind()
    dev = _device("W", W)
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_int_gemm, A, a_scales, W, w_scales, Y, bias, workspace, stream)
    raw = _raw(dev, stream)
    T = A.shape[0]
    M, K, ldw, ldy, dt, sp, bp = _product(W, w_scales, Y, T, bias, dev)
    if A.dtype is not torch.int8 or A.get_device() != dev:
        raise ValueError("A must be an int8 device tensor on W's device")
    lda = _rows("A", A, T, K, _pad16(K))
    if workspace is None:
        workspace = _workspace(bcq_int_workspace_bytes(T, M, K), W.device, stream)
    r = lib.bcq_int_gemm(A.data_ptr(), _plain("a_scales", a_scales, torch.float32, (T,), dev), T,
                         lda, W.data_ptr(), sp, M, K, ldw, bp, Y.data_ptr(), ldy, dt,
                         *_space(workspace, dev), raw)
    if r:
        _fail("bcq_int_gemm", r)


def bcq_int_linear(X, W, w_scales, Y, bias=None, workspace=None, stream=None) -> None:
    """``Y = X W^T + bias`` with the tokens ``X`` [T][K] rounded to 8 bits on the way and ``W``
    [M][K] held in 8 bits with the scales ``w_scales`` [M] (see ``include/bcq.h``).

    ``workspace=None`` allocates one through torch; :func:`new_int_workspace` keeps that out of
    a hot loop."""
    lib = _lib or _bind()
    dev = _device("W", W)
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_int_linear, X, W, w_scales, Y, bias, workspace, stream)
    raw = _raw(dev, stream)
    T = X.shape[0]
    M, K, ldw, ldy, dt, sp, bp = _product(W, w_scales, Y, T, bias, dev)
    if X.dtype is not Y.dtype or X.get_device() != dev:
        raise ValueError("X and Y must be device tensors of one dtype on W's device")
    ldx = _rows("X", X, T, K, K)
    if T == 1:
        ldx = _pad16(ldx)  # a single row has no next one to be aligned with
    if workspace is None:
        workspace = _workspace(bcq_int_workspace_bytes(T, M, K), W.device, stream)
    r = lib.bcq_int_linear(X.data_ptr(), T, ldx, W.data_ptr(), sp, M, K, ldw, bp, Y.data_ptr(),
                           ldy, dt, *_space(workspace, dev), raw)
    if r:
        _fail("bcq_int_linear", r)


# ----------------------------------------------------------------------------- norm


def bcq_rms_norm(X, gamma, eps, residual=None, H=None, Y=None, codes=None, scales=None,
                 stream=None) -> None:
    """``h = X + residual`` into ``H``, its root-mean-square norm times ``gamma`` [K] into ``Y``,
    and that rounded to 8 bits into ``codes`` (int8 [T][K], rows padded to 16 bytes) and
    ``scales`` (float32 [T]), as :func:`bcq_int_gemm` reads them; what is None is left out.
    All rows are [T][K] of ``X``'s dtype, 16-byte aligned; ``H`` may be ``X`` or ``residual``."""
    lib = _lib or _bind()
    dev = _device("X", X)
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_rms_norm, X, gamma, eps, residual, H, Y, codes, scales, stream)
    raw = _raw(dev, stream)
    dt, shape, dtype = _float("X", X, dev), X.shape, X.dtype
    if len(shape) != 2:
        raise ValueError("X must be [T][K], got %s" % (tuple(shape),))
    T, K = shape
    xp, ldx = _like("X", X, shape, dtype, dev)
    rp, ldr = (0, 0) if residual is None else _like("residual", residual, shape, dtype, dev)
    hp, ldh = (0, 0) if H is None else _like("H", H, shape, dtype, dev)
    yp, ldy = (0, 0) if Y is None else _like("Y", Y, shape, dtype, dev)
    cp = ldc = sp = 0
    if codes is not None:
        if codes.dtype is not torch.int8 or codes.get_device() != dev:
            raise ValueError("codes must be an int8 device tensor on X's device")
        cp, ldc = codes.data_ptr(), _rows("codes", codes, T, K, _pad16(K))
    if scales is not None:
        sp = _plain("scales", scales, torch.float32, (T,), dev)
    r = lib.bcq_rms_norm(xp, ldx, rp, ldr, _plain("gamma", gamma, dtype, (K,), dev), eps, T, K, dt,
                         hp, ldh, yp, ldy, cp, ldc, sp, raw)
    if r:
        _fail("bcq_rms_norm", r)


# ----------------------------------------------------------------------------- 4-bit cache


class KVCache:
    """A paged 4-bit key/value cache and its ``bcq_kv_cache`` descriptor.

    ``k_codes`` uint8 [pages][heads][page][D/2], ``v_codes`` uint8 [pages][heads][page/4][2D],
    ``scales`` float16 [pages][heads][page][4], ``page_table`` int32 [batch][max_pages] and
    ``lens`` int32 [batch], all on one device.  The tensors are the caller's and may be
    changed in place; the descriptor holds their addresses."""

    def __init__(self, k_codes, v_codes, scales, page_table, lens):
        _lib or _bind()
        if k_codes.dim() != 4 or page_table.dim() != 2:
            raise ValueError("k_codes must be [pages][heads][page][D/2] and page_table 2-D")
        P, H, page, half = k_codes.shape
        D = 2 * half
        B, width = page_table.shape
        dev = self._dev = _device("k_codes", k_codes)
        self._st = _KVCache(
            B, H, D, page, P, width,
            _plain("k_codes", k_codes, torch.uint8, (P, H, page, half), dev),
            _plain("v_codes", v_codes, torch.uint8, (P, H, page // 4, 2 * D), dev),
            _plain("scales", scales, torch.float16, (P, H, page, 4), dev),
            _plain("page_table", page_table, torch.int32, (B, width), dev),
            _plain("lens", lens, torch.int32, (B,), dev))
        self._ref = ctypes.byref(self._st)
        self.k_codes, self.v_codes, self.scales = k_codes, v_codes, scales
        self.page_table, self.lens = page_table, lens
        self.batch, self.heads, self.head_dim, self.page_tokens = B, H, D, page
        self.room, self.num_pages = width * page, P
        self._slots = (B, H, self.room)  # of weights and positions

    @classmethod
    def new(cls, batch: int, tokens: int, heads: int, head_dim: int, page_tokens: int = 64,
            device="cuda") -> "KVCache":
        """An empty cache with room for `tokens` tokens of each sequence, pages in order."""
        _lib or _bind()
        width = -(-tokens // page_tokens)
        P = batch * width
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)  # noqa: E731
        return cls(z((P, heads, page_tokens, head_dim // 2), torch.uint8),
                   z((P, heads, page_tokens // 4, 2 * head_dim), torch.uint8),
                   z((P, heads, page_tokens, 4), torch.float16),
                   torch.arange(P, dtype=torch.int32, device=device).view(batch, width),
                   z((batch,), torch.int32))

    @classmethod
    def pool(cls, batch: int, tokens: int, pages: int, heads: int, head_dim: int,
             page_tokens: int = 64, device="cuda"):
        """``(cache, free_pages, free_count)`` for :func:`bcq_kv_reserve`: `pages` pages, all of
        them free, and empty tables with room for `tokens` tokens of each of `batch` sequences."""
        _lib or _bind()
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)  # noqa: E731
        cache = cls(z((pages, heads, page_tokens, head_dim // 2), torch.uint8),
                    z((pages, heads, page_tokens // 4, 2 * head_dim), torch.uint8),
                    z((pages, heads, page_tokens, 4), torch.float16),
                    torch.full((batch, -(-tokens // page_tokens)), -1, dtype=torch.int32,
                               device=device),
                    z((batch,), torch.int32))
        # the lowest on top
        return (cache, torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                torch.full((1,), pages, dtype=torch.int32, device=device))

    def tracking(self):
        """Zeroed ``(weights, pos)`` for this cache, as append, attend and evict take them."""
        return (torch.zeros(self._slots, dtype=torch.float32, device=self.lens.device),
                torch.zeros(self._slots, dtype=torch.int32, device=self.lens.device))

    def ref(self):
        return self._ref


def _pair(K, V, cache: KVCache):
    """(n, dtype, strides of K, of V) of vectors [batch][n][heads][D] with contiguous channels."""
    shape = K.shape
    if len(shape) != 4 or shape[0] != cache.batch or shape[2] != cache.heads or \
            shape[3] != cache.head_dim or V.shape != shape:
        raise ValueError("K and V must be [%d][n][%d][%d], got %s and %s" %
                         (cache.batch, cache.heads, cache.head_dim, tuple(shape),
                          tuple(V.shape)))
    dt = _float("K", K, cache._dev)
    if V.dtype is not K.dtype or V.get_device() != cache._dev:
        raise ValueError("K and V must be device tensors of one dtype on the cache's device")
    ks, vs = K.stride(), V.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("K and V must have contiguous channels")
    return shape[1], dt, ks, vs


def bcq_kv_append(cache: KVCache, K, V, positions=None, weights=None, pos=None,
                  stream=None) -> None:
    """Quantizes ``K`` and ``V`` [batch][n][heads][D] into the last n slots of every sequence;
    ``cache.lens`` must count them already.  ``weights`` and ``pos`` [batch][heads][room] get 0
    and the token's position (``positions`` int32 [batch][n], or its slot)."""
    dev, slots = cache._dev, cache._slots
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_append, cache, K, V, positions, weights, pos, stream)
    n, dt, ks, vs = _pair(K, V, cache)
    r = _lib.bcq_kv_append(
        cache._ref, n, K.data_ptr(), ks[0], ks[1], ks[2], V.data_ptr(), vs[0], vs[1], vs[2], dt,
        0 if positions is None else _plain("positions", positions, torch.int32,
                                           (cache.batch, n), dev),
        0 if weights is None else _plain("weights", weights, torch.float32, slots, dev),
        0 if pos is None else _plain("pos", pos, torch.int32, slots, dev), _raw(dev, stream))
    if r:
        _fail("bcq_kv_append", r)


def bcq_kv_read(cache: KVCache, K, V, stream=None) -> None:
    """Writes the values of the last n cached tokens to ``K`` and ``V`` [batch][n][heads][D]."""
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_read, cache, K, V, stream)
    n, dt, ks, vs = _pair(K, V, cache)
    r = _lib.bcq_kv_read(cache._ref, n, K.data_ptr(), ks[0], ks[1], ks[2], V.data_ptr(), vs[0],
                         vs[1], vs[2], dt, _raw(dev, stream))
    if r:
        _fail("bcq_kv_read", r)


def bcq_kv_reserve_workspace_bytes(cache: KVCache) -> int:
    return int(_lib.bcq_kv_reserve_workspace_bytes(cache._ref))


def new_kv_reserve_workspace(cache: KVCache):
    """A device workspace for :func:`bcq_kv_reserve`; calls that may overlap need separate ones."""
    return _workspace(bcq_kv_reserve_workspace_bytes(cache), cache.lens.device, None)


def bcq_kv_reserve(cache: KVCache, new_tokens, free_pages, free_count, starts, slots, positions,
                   release=None, shared_pages: int = 0, lens_out=None, page_table_out=None,
                   free_pages_out=None, free_count_out=None, workspace=None, stream=None) -> None:
    """Takes back the pages of the sequences that ended (``release`` int32 [batch], or None) and
    gives pages for ``new_tokens`` int32 [batch] from the stack ``free_pages`` int32 [pages] of
    ``free_count`` int32 [1].  Writes ``starts`` int32 [batch + 1] and, for T packed tokens,
    ``slots`` int64 [T] and ``positions`` int32 [T]; the cache's lengths and table and the stack
    in place unless the ``_out`` arrays are given (see ``include/bcq.h``)."""
    dev, i32 = cache._dev, torch.int32
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_reserve, cache, new_tokens, free_pages, free_count, starts,
                      slots, positions, release, shared_pages, lens_out, page_table_out,
                      free_pages_out, free_count_out, workspace, stream)
    raw, B, T = _raw(dev, stream), (cache.batch,), slots.shape
    stack = (cache.num_pages,)
    free = _plain("free_pages", free_pages, i32, stack, dev)
    count = _plain("free_count", free_count, i32, (1,), dev)
    if len(T) != 1:
        raise ValueError("slots must be [T], got %s" % (tuple(T),))
    if workspace is None:
        workspace = _workspace(bcq_kv_reserve_workspace_bytes(cache), cache.lens.device, stream)
    r = _lib.bcq_kv_reserve(
        cache._ref, _plain("new_tokens", new_tokens, i32, B, dev),
        0 if release is None else _plain("release", release, i32, B, dev), shared_pages, free,
        count, T[0],
        cache._st.lens if lens_out is None else _plain("lens_out", lens_out, i32, B, dev),
        cache._st.page_table if page_table_out is None
        else _plain("page_table_out", page_table_out, i32, cache.page_table.shape, dev),
        free if free_pages_out is None
        else _plain("free_pages_out", free_pages_out, i32, stack, dev),
        count if free_count_out is None
        else _plain("free_count_out", free_count_out, i32, (1,), dev),
        _plain("starts", starts, i32, (cache.batch + 1,), dev),
        _plain("slots", slots, torch.int64, T, dev), _plain("positions", positions, i32, T, dev),
        *_space(workspace, dev), raw)
    if r:
        _fail("bcq_kv_reserve", r)


def _packed(K, V, slots, cache: KVCache):
    """(T, dtype, strides of K, of V) of packed vectors [T][heads][D] with contiguous channels."""
    shape = K.shape
    if len(shape) != 3 or shape[1] != cache.heads or shape[2] != cache.head_dim or \
            V.shape != shape:
        raise ValueError("K and V must be [T][%d][%d], got %s and %s" %
                         (cache.heads, cache.head_dim, tuple(shape), tuple(V.shape)))
    dt = _float("K", K, cache._dev)
    if V.dtype is not K.dtype or V.get_device() != cache._dev:
        raise ValueError("K and V must be device tensors of one dtype on the cache's device")
    ks, vs = K.stride(), V.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("K and V must have contiguous channels")
    return shape[0], dt, ks, vs, _plain("slots", slots, torch.int64, shape[:1], cache._dev)


def bcq_kv_append_slots(cache: KVCache, K, V, slots, stream=None) -> None:
    """Quantizes packed ``K`` and ``V`` [T][heads][D] into the slots ``slots`` int64 [T], as
    :func:`bcq_kv_reserve` writes them."""
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_append_slots, cache, K, V, slots, stream)
    T, dt, ks, vs, sp = _packed(K, V, slots, cache)
    r = _lib.bcq_kv_append_slots(cache._ref, T, sp, K.data_ptr(), ks[0], ks[1], V.data_ptr(),
                                 vs[0], vs[1], dt, _raw(dev, stream))
    if r:
        _fail("bcq_kv_append_slots", r)


def bcq_kv_read_slots(cache: KVCache, K, V, slots, stream=None) -> None:
    """Writes the values cached in ``slots`` int64 [T] to ``K`` and ``V`` [T][heads][D]."""
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_read_slots, cache, K, V, slots, stream)
    T, dt, ks, vs, sp = _packed(K, V, slots, cache)
    r = _lib.bcq_kv_read_slots(cache._ref, T, sp, K.data_ptr(), ks[0], ks[1], V.data_ptr(), vs[0],
                               vs[1], dt, _raw(dev, stream))
    if r:
        _fail("bcq_kv_read_slots", r)


def bcq_kv_workspace_bytes(cache: KVCache, n: int, q_heads: int, with_weights: bool) -> int:
    return int(_lib.bcq_kv_workspace_bytes(cache._ref, n, q_heads, bool(with_weights)))


def new_kv_workspace(cache: KVCache, n: int, q_heads: int, weights: bool = False):
    """A device workspace for :func:`bcq_kv_attend` with n queries a sequence; calls that may
    overlap need separate ones."""
    return _workspace(bcq_kv_workspace_bytes(cache, n, q_heads, weights), cache.lens.device,
                      None)


def bcq_kv_attend(cache: KVCache, Q, O, scale=None, weights=None, workspace=None,
                  stream=None) -> None:
    """Causal attention of ``Q`` [batch][n][q_heads][D], the queries of the last n cached tokens,
    over the cache into ``O`` (same shape); ``scale`` defaults to 1/sqrt(D).  ``weights``
    [batch][heads][room] float32 accumulates each cached token's probabilities."""
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_attend, cache, Q, O, scale, weights, workspace, stream)
    raw = _raw(dev, stream)
    dt = _float("Q", Q, dev)
    shape = Q.shape
    if len(shape) != 4 or shape[0] != cache.batch or shape[3] != cache.head_dim or \
            O.shape != shape or O.dtype is not Q.dtype or O.get_device() != dev:
        raise ValueError("Q and O must be [%d][n][q_heads][%d] of one dtype on the cache's device" %
                         (cache.batch, cache.head_dim))
    n, heads = shape[1], shape[2]
    qs, os = Q.stride(), O.stride()
    if qs[3] != 1 or os[3] != 1:
        raise ValueError("Q and O must have contiguous channels")
    if workspace is None:
        workspace = _workspace(bcq_kv_workspace_bytes(cache, n, heads, weights is not None),
                               Q.device, stream)
    r = _lib.bcq_kv_attend(
        cache._ref, Q.data_ptr(), n, heads, qs[0], qs[1], qs[2], O.data_ptr(), os[0], os[1],
        os[2], dt, shape[3] ** -0.5 if scale is None else scale,
        0 if weights is None else _plain("weights", weights, torch.float32, cache._slots, dev),
        *_space(workspace, dev), raw)
    if r:
        _fail("bcq_kv_attend", r)


def bcq_kv_packed_workspace_bytes(cache: KVCache, T: int, q_heads: int, max_n: int,
                                  shared_pages: int = 0) -> int:
    return int(_lib.bcq_kv_packed_workspace_bytes(cache._ref, T, q_heads, max_n, shared_pages))


def new_kv_packed_workspace(cache: KVCache, T: int, q_heads: int, max_n: int,
                            shared_pages: int = 0):
    """A device workspace for :func:`bcq_kv_attend_packed`; calls that may overlap need separate
    ones."""
    return _workspace(bcq_kv_packed_workspace_bytes(cache, T, q_heads, max_n, shared_pages),
                      cache.lens.device, None)


def bcq_kv_attend_packed(cache: KVCache, Q, O, starts, max_n: int, shared_pages: int = 0,
                         scale=None, workspace=None, stream=None) -> None:
    """Causal attention of packed tokens ``Q`` [T][q_heads][D], ``starts[b]`` to
    ``starts[b + 1]`` (int32 [batch + 1]) the last of sequence b and at most ``max_n`` of each,
    over the cache into ``O`` (same shape).  The first ``shared_pages`` entries of every
    sequence's table are the same.  ``scale`` defaults to 1/sqrt(D)."""
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_attend_packed, cache, Q, O, starts, max_n, shared_pages, scale,
                      workspace, stream)
    raw = _raw(dev, stream)
    dt = _float("Q", Q, dev)
    shape = Q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim or O.shape != shape or \
            O.dtype is not Q.dtype or O.get_device() != dev:
        raise ValueError("Q and O must be [T][q_heads][%d] of one dtype on the cache's device" %
                         cache.head_dim)
    qs, os = Q.stride(), O.stride()
    if qs[2] != 1 or os[2] != 1:
        raise ValueError("Q and O must have contiguous channels")
    if workspace is None:
        workspace = _workspace(
            bcq_kv_packed_workspace_bytes(cache, shape[0], shape[1], max_n, shared_pages),
            Q.device, stream)
    r = _lib.bcq_kv_attend_packed(
        cache._ref, Q.data_ptr(), shape[0], shape[1], qs[0], qs[1],
        _plain("starts", starts, torch.int32, (cache.batch + 1,), dev), max_n, shared_pages,
        O.data_ptr(), os[0], os[1], dt, shape[2] ** -0.5 if scale is None else scale,
        *_space(workspace, dev), raw)
    if r:
        _fail("bcq_kv_attend_packed", r)


def bcq_kv_evict_workspace_bytes(cache: KVCache, keep: int) -> int:
    return int(_lib.bcq_kv_evict_workspace_bytes(cache._ref, keep))


def new_kv_evict_workspace(cache: KVCache, keep: int):
    """A device workspace for :func:`bcq_kv_evict`; calls that may overlap need separate ones."""
    return _workspace(bcq_kv_evict_workspace_bytes(cache, keep), cache.lens.device, None)


def bcq_kv_evict(cache: KVCache, keep: int, recent: int, weights, pos, lens_out=None,
                 weights_out=None, pos_out=None, workspace=None, stream=None) -> None:
    """Shrinks every sequence to at most ``keep`` tokens a head, the ``recent`` newest and those of
    the largest ``weights``.  In place unless ``lens_out``, ``weights_out``, ``pos_out`` are
    given (the codes always are: see ``include/bcq.h``)."""
    slots, f32, i32 = cache._slots, torch.float32, torch.int32
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        return _there(dev, bcq_kv_evict, cache, keep, recent, weights, pos, lens_out, weights_out,
                      pos_out, workspace, stream)
    raw = _raw(dev, stream)
    w, p = _plain("weights", weights, f32, slots, dev), _plain("pos", pos, i32, slots, dev)
    if workspace is None:
        workspace = _workspace(bcq_kv_evict_workspace_bytes(cache, keep), weights.device, stream)
    r = _lib.bcq_kv_evict(
        cache._ref, keep, recent, w, p,
        cache.lens.data_ptr() if lens_out is None
        else _plain("lens_out", lens_out, i32, (cache.batch,), dev),
        w if weights_out is None else _plain("weights_out", weights_out, f32, slots, dev),
        p if pos_out is None else _plain("pos_out", pos_out, i32, slots, dev),
        *_space(workspace, dev), raw)
    if r:
        _fail("bcq_kv_evict", r)
