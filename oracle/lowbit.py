"""Float64 definitions of the low-bit serving operators on host arrays: the 8-bit rows and
their product, the 4-bit key/value vectors, their pages, attention and eviction.  Test
infrastructure only; it shares no code with the library."""

from __future__ import annotations

import numpy as np

# ------------------------------------------------------------------------------ 8-bit rows


def quantize_rows(x):
    """(codes int8, scales float32) of each row: the scale (a product with the constant 1/127)
    and the codes (a quotient, halves to even) are defined in single precision."""
    x = np.asarray(x).astype(np.float32)
    with np.errstate(invalid="ignore"):
        top = np.abs(x).max(axis=1)
        scale = np.where(top < np.inf, top * np.float32(1 / 127), np.float32(np.nan))
        scale = scale.astype(np.float32)
        good = (scale > 0) & np.isfinite(scale)
        q = np.rint(x / np.where(good, scale, np.float32(1))[:, None])
    q = np.where(good[:, None], q, 0)
    return np.clip(q, -127, 127).astype(np.int8), scale


def product(codes, scales, w, w_scales, bias=None):
    """sum_k codes w, times both scales, plus the bias, in float64."""
    y = (codes.astype(np.int64) @ w.astype(np.int64).T).astype(np.float64)
    y = y * scales.astype(np.float64)[:, None] * w_scales.astype(np.float64)[None]
    return y if bias is None else y + bias.astype(np.float64)


# ------------------------------------------------------------------------------ 4-bit vectors


def quantize_vectors(x):
    """(codes uint8, scale float16, zero float16) along the last axis, as the format says."""
    x = np.asarray(x).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        lo, hi = x.min(axis=-1), x.max(axis=-1)
        scale = ((hi - lo) * np.float32(1 / 15)).astype(np.float16)
        zero = lo.astype(np.float16)
        scale = np.where(np.isfinite(scale) & np.isfinite(zero), scale, np.float16(np.nan))
        s = scale.astype(np.float32)[..., None]
        q = np.where(s > 0, (x - zero.astype(np.float32)[..., None]) / np.where(s > 0, s, 1), 0)
        q = np.nan_to_num(np.rint(q), nan=0, posinf=15, neginf=0)
    return np.clip(q, 0, 15).astype(np.uint8), scale, zero


def k_bytes(codes):
    """Codes [..., D] of one token's key as its D/2 bytes."""
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def v_place(D):
    """(byte within a block of 4 tokens for token 0, shift) of every channel of V."""
    d = np.arange(D)
    byte = (d % 64) // 4 * (D // 8) + d // 64 * 8 + (d % 4) // 2
    return byte, d % 2 * 4


class Cache:
    """A cache in the library's byte layout on the host."""

    def __init__(self, pages, heads, page, D, table, lens):
        self.k = np.zeros((pages, heads, page, D // 2), np.uint8)
        self.v = np.zeros((pages, heads, page // 4, 2 * D), np.uint8)
        self.s = np.zeros((pages, heads, page, 4), np.float16)
        self.table, self.lens = np.asarray(table, np.int32), np.asarray(lens, np.int32)
        self.H, self.page, self.D = heads, page, D

    def put(self, b, h, slot, k, v):
        """Quantizes one token's key and value [D] into a slot."""
        p, line = self.table[b, slot // self.page], slot % self.page
        ck, sk, zk = quantize_vectors(k)
        cv, sv, zv = quantize_vectors(v)
        self.k[p, h, line] = k_bytes(ck)
        byte, shift = v_place(self.D)
        block = self.v[p, h, line // 4]
        at = byte + line % 4 * 2
        for half in (0, 4):
            sel = shift == half
            block[at[sel]] = (block[at[sel]] & ~np.uint8(15 << half)) | (cv[sel] << half)
        self.s[p, h, line] = [sk, zk, sv, zv]

    def get(self, b, h, slots):
        """(keys, values, scales) [len(slots)][D] in float64, [len(slots)][4]."""
        slots = np.asarray(slots, np.int64)
        p, line = self.table[b, slots // self.page], slots % self.page
        s = self.s[p, h, line].astype(np.float64)
        d = np.arange(self.D)
        ck = self.k[p, h, line][:, d // 2] >> (d % 2 * 4) & 15
        byte, shift = v_place(self.D)
        at = byte[None] + (line % 4 * 2)[:, None]
        cv = np.take_along_axis(self.v[p, h, line // 4], at, 1) >> shift & 15
        return s[:, 1:2] + s[:, 0:1] * ck, s[:, 3:4] + s[:, 2:3] * cv, s


def attend(cache, q, scale):
    """(out, probabilities) in float64: q [B][n][Hq][D]; probabilities [B][H][longest] are the
    sums over the queries and over the query heads of a cached head.  With them what errors are
    bounded by: for outputs (terms of the scores that the probabilities carry over, terms that
    a rounding of probability times V scale acts on, the same for roundings at the row's largest
    term), for probabilities the terms of the scores."""
    q = np.asarray(q).astype(np.float64)
    B, n, Hq, D = q.shape
    G = Hq // cache.H
    out = np.zeros_like(q)
    T = int(cache.lens.max(initial=0))
    total = np.zeros((B, cache.H, max(T, 0)))
    bounds = np.zeros((3,) + q.shape)
    wbound = np.zeros_like(total)
    for b in range(B):
        L = int(cache.lens[b])
        for h in range(cache.H):
            if L <= 0:
                continue
            k, v, s = cache.get(b, h, np.arange(L))
            with np.errstate(invalid="ignore"):
                ck = np.where(s[:, 0:1] > 0, (k - s[:, 1:2]) / s[:, 0:1], 0)
            for i in range(n):
                m = L - n + i + 1
                if m <= 0:
                    continue
                for g in range(h * G, (h + 1) * G):
                    x = q[b, i, g]
                    z = scale * (k[:m] @ x)
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    out[b, i, g] = p @ v[:m]
                    total[b, h, :m] += p
                    # |terms| a score is summed from, and what they weigh in an output
                    mag = abs(scale) * (s[:m, 0] * (np.abs(x) @ ck[:m].T)
                                        + np.abs(s[:m, 1]) * np.abs(x).sum())
                    bounds[0, b, i, g] = mag.max() * (p @ np.abs(v[:m]) + np.abs(out[b, i, g]))
                    top = (p * s[:m, 2]).max()
                    bounds[1, b, i, g] = p @ np.abs(v[:m] - s[:m, 3:4])
                    bounds[2, b, i, g] = 15 * m * top
                    wbound[b, h, :m] += p * mag.max()
    return out, total, bounds, wbound


# ------------------------------------------------------------------------------ eviction


def kept_slots(length, keep, recent, weights, pos):
    """The sorted slots that a head keeps."""
    if length <= keep:
        return np.arange(length)
    w, p = weights[:length].astype(np.float64), pos[:length].astype(np.int64)
    late = p > p.max() - recent
    w = np.where(np.isnan(w), -np.inf, w)
    nan = np.isnan(weights[:length])
    order = sorted(range(length), key=lambda t: (not late[t], bool(nan[t]), -w[t], t))
    return np.sort(order[:keep])


def evict(length, keep, recent, weights, pos):
    """Where each remaining slot's token comes from."""
    kept = kept_slots(length, keep, recent, weights, pos)
    m = min(length, keep)
    src = np.arange(m)
    held = set(kept.tolist())
    holes = [t for t in range(m) if t not in held]
    fill = [t for t in kept.tolist() if t >= m]
    src[holes] = fill
    return src
