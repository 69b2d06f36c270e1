"""Binding of the low-bit serving operators: the 8-bit integer linear layer and the 4-bit
key/value cache (append, read, attend, evict).  Names and semantics are those of
``include/bcq.h``; the package exports everything here.

The tensors of a call, and its ``stream`` if one is given, belong to one device, which need not be
the current one.
"""

from __future__ import annotations

import ctypes

BCQ_KV_MAX_TOKENS = 1 << 24

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
    "bcq_kv_append": (_int, [_kc, _i32, _vp, *_strides, _vp, *_strides, _int, _vp, _vp, _vp,
                             _vp]),
    "bcq_kv_read": (_int, [_kc, _i32, _vp, *_strides, _vp, *_strides, _int, _vp]),
    "bcq_kv_attend": (_int, [_kc, _vp, _i32, _i32, *_strides, _vp, *_strides, _int,
                             ctypes.c_float, _vp, _vp, _sz, _vp]),
    "bcq_kv_workspace_bytes": (_sz, [_kc, _i32, _i32, _i32]),
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
        self.room = width * page
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
