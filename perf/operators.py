"""The low-bit serving operators, as they are measured: an 8-bit integer linear layer, and a
key/value cache held in 4 bits with the quantizer that fills it, the attention that reads it and
the eviction that shrinks it by accumulated attention weight.

``run(state)`` is one pass: the plain form of torch operations in 32 bits where ``own`` is False,
the library's entry points where it is True.  Both take the same state and return the same
outputs.  ``exact(case, seed)`` is the definition in 64 bits.

Formats (bytes as the library defines them):

* 8-bit rows: code = rint(x / s), s = max|x| / 127 for each row; value = s * code.
* 4-bit vectors: one fp16 scale and one fp16 zero for each (token, head, K or V) vector of D
  channels; zero = min, scale = (max - min) / 15, code = clamp(rint((x - zero) / scale), 0, 15);
  value = zero + scale * code.
* Pages of ``page`` tokens: K codes [pages][heads][page][D/2], two channels a byte, the even one
  in the low half; V codes [pages][heads][page/4][16][D/64][4][2]: blocks of four tokens, in a
  block byte (r, h, t, c) holds channels 64h + 4r + 2c and + 1 of its token t; scales
  [pages][heads][page][4] = (K scale, K zero, V scale, V zero).
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # one token through a 4096 x 4096 projection: the latency of a decode step's smallest product
        {"name": "linear 1x4096x4096 f16", "op": "linear", "dtype": "f16", "tokens": 1,
         "rows": 4096, "cols": 4096, "bias": False},
        # a batch of decode requests, not a whole tile of them, through the gate projection
        {"name": "linear 37x14336x4096 f16", "op": "linear", "dtype": "f16", "tokens": 37,
         "rows": 14336, "cols": 4096, "bias": False},
        # odd sizes in every direction, single precision, with a bias
        {"name": "linear 515x1000x1001 f32", "op": "linear", "dtype": "f32", "tokens": 515,
         "rows": 1000, "cols": 1001, "bias": True},
        # a prompt of 4096 tokens through the gate projection: bound by the matrix cores
        {"name": "linear 4096x14336x4096 f16", "op": "linear", "dtype": "f16", "tokens": 4096,
         "rows": 14336, "cols": 4096, "bias": False},
        # one new token of each of 64 sequences enters the cache
        {"name": "append 64x1 f16", "op": "append", "dtype": "f16", "batch": 64, "tokens": 1,
         "kv_heads": 8, "dim": 128, "page": 64, "context": 1500},
        # two prompts of an odd length enter it, in single precision and small pages
        {"name": "append 2x4099 f32", "op": "append", "dtype": "f32", "batch": 2, "tokens": 4099,
         "kv_heads": 8, "dim": 64, "page": 16, "context": 4099},
        # a single request's decode step on a short context: latency
        {"name": "attend 1x1 ctx 1023 f16", "op": "attend", "dtype": "f16", "batch": 1,
         "queries": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "context": 1023,
         "weights": False},
        # a serving batch's decode step with the weights that eviction goes by
        {"name": "attend 32x1 ctx 8192 f16 w", "op": "attend", "dtype": "f16", "batch": 32,
         "queries": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "context": 8192,
         "weights": True},
        # drafted tokens checked in one pass: every head with its own keys, single precision
        {"name": "attend 3x5 ctx 3001 f32 w", "op": "attend", "dtype": "f32", "batch": 3,
         "queries": 5, "heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "context": 3001,
         "weights": True},
        # a chunk of two long prompts against what is cached already
        {"name": "attend 2x2048 ctx 6001 f16", "op": "attend", "dtype": "f16", "batch": 2,
         "queries": 2048, "heads": 32, "kv_heads": 8, "dim": 128, "page": 128, "context": 6001,
         "weights": False},
        # a decode loop at its budget: every step one token too many in each head
        {"name": "evict 32x2049 to 2048", "op": "evict", "batch": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "length": 2049, "keep": 2048, "recent": 64},
        # long prompts cut down once, after they were read
        {"name": "evict 4x32768 to 4096", "op": "evict", "batch": 4, "kv_heads": 8, "dim": 128,
         "page": 64, "length": 32768, "keep": 4096, "recent": 512},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (16, 16), (28, 4), (8, 1), (12, 12), (64, 8), (40, 8)]


def draw(rng):
    op = rng.choice(["linear", "linear", "append", "attend", "attend", "attend", "evict"])
    dtype = rng.choice(["f16", "f16", "f32"])
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    if op == "linear":
        tokens, rows = _log(rng, 1, 4096), _log(rng, 64, 14336)
        cols = _log(rng, 65, 14336)
        rows = min(rows, max(1, 4096 * 14336 * 4096 // (tokens * cols)))
        return {"op": op, "dtype": dtype, "tokens": tokens, "rows": rows, "cols": cols,
                "bias": rng.random() < 0.5}
    if op == "append":
        batch, kv_heads = _log(rng, 1, 64), rng.choice([1, 4, 8, 16])
        tokens = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 8192 // batch))
        return {"op": op, "dtype": dtype, "batch": batch, "tokens": tokens, "kv_heads": kv_heads,
                "dim": dim, "page": page, "context": tokens + _log(rng, 1, 2000)}
    if op == "attend":
        heads, kv_heads = rng.choice(HEADS)
        if rng.random() < 0.6:  # decode: one token, or a few drafted ones
            queries = rng.choice([1, 1, 1, 2, 5, 8])
            batch = _log(rng, 1, 32)
            context = _log(rng, 9, max(9, min(131072, 262144 * 8 // (batch * max(8, kv_heads)))))
        else:
            queries, batch = _log(rng, 17, 2048), rng.choice([1, 2])
            context = queries + _log(rng, 1, 4000)
            most = 2 * 2048 * 6001 * 32 * 128
            queries = min(queries, most // (batch * context * heads * dim))
        return {"op": op, "dtype": dtype, "batch": batch, "queries": queries, "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "page": page, "context": context,
                "weights": rng.random() < 0.5}
    length = _log(rng, 100, 32768)
    keep = length - 1 if rng.random() < 0.4 else _log(rng, 16, length)
    return {"op": op, "batch": _log(rng, 1, max(1, 131072 // length)), "kv_heads":
            rng.choice([1, 4, 8]), "dim": dim, "page": page, "length": length, "keep": keep,
            "recent": min(keep, _log(rng, 1, 512))}


def _lengths(batch, longest):
    """Sequences of unlike lengths, from the longest down to about half of it."""
    return [longest - i * (longest // 2) // batch for i in range(batch)]


# ------------------------------------------------------------------------------ inputs


def _pad(n, m):
    return (n + m - 1) // m * m


def _four_bits(x):
    """(codes, scale, zero) of vectors along the last dimension, as the library's format says."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale, zero = ((hi - lo) / 15).half(), lo.half()
    s = scale.float()
    q = torch.where(s > 0, (x - zero.float()) / torch.where(s > 0, s, 1.0), 0.0)
    return torch.round(q).clamp(0, 15).to(torch.uint8), scale, zero


def _pack_v(codes):
    P, H, T, D = codes.shape
    c = codes.view(P, H, T // 4, 4, D // 64, 16, 2, 2)
    b = c[..., 0] | c[..., 1] << 4  # [P][H][T/4][t][h][r][c]
    return b.permute(0, 1, 2, 5, 4, 3, 6).reshape(P, H, T // 4, 2 * D).contiguous()


def _cache(case, lens, room, g):
    """Random keys and values in 4 bits in scattered pages, tables of `room` tokens a sequence."""
    page, H, D = case["page"], case["kv_heads"], case["dim"]
    B, width = len(lens), _pad(room, page) // page
    pages = B * width
    k = torch.randn((pages, H, page, D), generator=g, device="cuda", dtype=torch.float16)
    k += torch.randn((1, H, 1, D), generator=g, device="cuda", dtype=torch.float16)  # channel means
    ck, sk, zk = _four_bits(k)
    del k
    v = torch.randn((pages, H, page, D), generator=g, device="cuda", dtype=torch.float16)
    cv, sv, zv = _four_bits(v)
    del v
    return {
        "k_codes": ck[..., 0::2] | ck[..., 1::2] << 4,
        "v_codes": _pack_v(cv),
        "scales": torch.cat([sk, zk, sv, zv], -1).contiguous(),
        "table": torch.randperm(pages, generator=g, device="cuda").int().view(B, width),
        "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
    }


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    state = {"case": dict(case)}
    dt = DTYPES[case.get("dtype", "f16")]
    if case["op"] == "linear":
        T, M, K = case["tokens"], case["rows"], case["cols"]
        # activations with a hundredth of the channels twenty times larger; rows start at 16 bytes
        x = torch.randn((T, _pad(K, 16)), generator=g, device="cuda")
        loud = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]
        x[:, loud] *= 20
        w = torch.randn((M, K), generator=g, device="cuda") * 0.02
        s = w.abs().amax(1) / 127
        codes = torch.zeros((M, _pad(K, 16)), dtype=torch.int8, device="cuda")
        codes[:, :K] = torch.round(w / s[:, None]).to(torch.int8)
        bias = torch.randn(M, generator=g, device="cuda").to(dt) if case["bias"] else None
        state.update(x=x.to(dt)[:, :K], w=codes[:, :K], w_scale=s, bias=bias,
                     y=torch.empty((T, M), dtype=dt, device="cuda"))
    elif case["op"] == "append":
        B, n, H, D = case["batch"], case["tokens"], case["kv_heads"], case["dim"]
        c = case["context"]
        state.update(_cache(case, _lengths(B, c) if c >= 2 * n else [c] * B, c, g))
        # keys and values lie behind the queries in one projection's output
        qkv = torch.randn((B, n, 4 * H, D), generator=g, device="cuda").to(dt)
        state.update(k=qkv[:, :, 2 * H:3 * H], v=qkv[:, :, 3 * H:],
                     k_out=torch.empty((B, n, H, D), dtype=dt, device="cuda"),
                     v_out=torch.empty((B, n, H, D), dtype=dt, device="cuda"))
    elif case["op"] == "attend":
        B, n, H = case["batch"], case["queries"], case["heads"]
        state.update(_cache(case, _lengths(B, case["context"]), case["context"], g))
        q = torch.randn((B, n, H, case["dim"]), generator=g, device="cuda").to(dt)
        state.update(q=q, out=torch.empty_like(q), weights=None)
        if case["weights"]:
            room = state["table"].shape[1] * case["page"]
            state["weights"] = torch.rand((B, case["kv_heads"], room), generator=g, device="cuda")
    else:
        B, H, L = case["batch"], case["kv_heads"], case["length"]
        state.update(_cache(case, [L] * B, L, g))
        room = state["table"].shape[1] * case["page"]
        w = torch.randn((B, H, room), generator=g, device="cuda").mul(2).exp()
        state.update(weights=w, pos=torch.arange(room, device="cuda").int().expand(B, H, room)
                     .contiguous(), weights_out=torch.zeros_like(w),
                     pos_out=torch.zeros((B, H, room), dtype=torch.int32, device="cuda"),
                     lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"))
    return state


# ------------------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "append": _own_append, "attend": _own_attend,
                "evict": _own_evict}[op](state)
    return {"linear": _linear, "append": _append, "attend": _attend, "evict": _evict}[op](state)


def _handle(bcq, s):
    """The cache's handle, made once, as a program keeps it with its cache."""
    h = s.get("handle")
    if h is None:
        h = s["handle"] = bcq.KVCache(s["k_codes"], s["v_codes"], s["scales"], s["table"],
                                      s["lens"])
    return h


def _own_linear(s):
    import binary_coded_precision_amd as bcq

    if "workspace" not in s:
        s["workspace"] = bcq.new_int_workspace(s["x"].shape[0], *s["w"].shape)
    bcq.bcq_int_linear(s["x"], s["w"], s["w_scale"], s["y"], bias=s["bias"],
                       workspace=s["workspace"])
    return s["y"]


def _own_append(s):
    import binary_coded_precision_amd as bcq

    h = _handle(bcq, s)
    bcq.bcq_kv_append(h, s["k"], s["v"])
    bcq.bcq_kv_read(h, s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


def _own_attend(s):
    import binary_coded_precision_amd as bcq

    h = _handle(bcq, s)
    if "workspace" not in s:
        s["workspace"] = bcq.new_kv_workspace(h, s["q"].shape[1], s["q"].shape[2],
                                              weights=s["weights"] is not None)
    bcq.bcq_kv_attend(h, s["q"], s["out"], weights=s["weights"], workspace=s["workspace"])
    return (s["out"],) if s["weights"] is None else (s["out"], s["weights"])


def _own_evict(s):
    import binary_coded_precision_amd as bcq

    h = _handle(bcq, s)
    if "workspace" not in s:
        s["workspace"] = bcq.new_kv_evict_workspace(h, s["case"]["keep"])
    bcq.bcq_kv_evict(h, s["case"]["keep"], s["case"]["recent"], s["weights"], s["pos"],
                     lens_out=s["lens_out"], weights_out=s["weights_out"], pos_out=s["pos_out"],
                     workspace=s["workspace"])
    return _evict_outputs(s)


# ------------------------------------------------------------------------------ plain forms


def _linear(s):
    x = s["x"].float()
    scale = x.abs().amax(1, keepdim=True) / 127
    codes = torch.round(x / torch.where(scale > 0, scale, 1.0))
    y = (codes @ s["w"].float().t()) * (scale * s["w_scale"])
    if s["bias"] is not None:
        y = y + s["bias"].float()
    s["y"].copy_(y)
    return s["y"]


def _nibbles(b):
    """Bytes [..., n] as the 2n codes they hold."""
    return torch.stack([b & 15, b >> 4], -1).flatten(-2).float()


def _unpack(s, pages):
    """Keys and values of the pages in 32 bits, [...][heads][page][D]."""
    sc = s["scales"][pages].float()
    k = _nibbles(s["k_codes"][pages]) * sc[..., 0:1] + sc[..., 1:2]
    D, T = k.shape[-1], k.shape[-2]
    v = s["v_codes"][pages].unflatten(-1, (16, D // 64, 4, 2))  # [...][T/4][r][h][t][c]
    v = v.movedim(-2, -4).transpose(-3, -2)  # [...][T/4][t][h][r][c]
    v = _nibbles(v).flatten(-3).flatten(-3, -2)  # [...][T][D]
    assert v.shape[-2] == T
    return k, v * sc[..., 2:3] + sc[..., 3:4]


def _whole(s):
    """Every sequence's keys and values in 32 bits, [batch][heads][room][D]."""
    k, v = _unpack(s, s["table"].long())  # [B][pages][H][page][D]
    return (t.transpose(1, 2).flatten(2, 3) for t in (k, v))


def _append(s):
    case = s["case"]
    n, page = case["tokens"], case["page"]
    slot = s["lens"].long()[:, None] - n + torch.arange(n, device="cuda")  # [B][n]
    at = torch.gather(s["table"].long(), 1, slot // page)
    ck, sk, zk = _four_bits(s["k"])
    cv, sv, zv = _four_bits(s["v"])
    # after the two indexes, the token's own dimensions: [B][n][H][...]
    s["k_codes"][at, :, slot % page] = ck[..., 0::2] | ck[..., 1::2] << 4
    D = case["dim"]
    v = cv.unflatten(-1, (D // 64, 16, 2, 2))
    v = (v[..., 0] | v[..., 1] << 4).transpose(-3, -2)  # [B][n][H][r][h][c]
    blocks = s["v_codes"].unflatten(-1, (16, D // 64, 4, 2))
    blocks[at, :, slot % page // 4, :, :, slot % 4] = v
    s["scales"][at, :, slot % page] = torch.cat([sk, zk, sv, zv], -1)
    # and read back as the values that they stand for
    c, m = _nibbles(s["k_codes"][at, :, slot % page]), s["scales"][at, :, slot % page].float()
    s["k_out"].copy_(c * m[..., 0:1] + m[..., 1:2])
    c = _nibbles(blocks[at, :, slot % page // 4, :, :, slot % 4].transpose(-3, -2)).flatten(-3)
    s["v_out"].copy_(c * m[..., 2:3] + m[..., 3:4])
    return s["k_out"], s["v_out"]


def _attend(s):
    q = s["q"].float()
    B, n, Hq, D = q.shape
    k, v = _whole(s)
    H, T = k.shape[1], k.shape[2]
    # rows of a cached head: its queries' heads, all the queries of each
    q = q.transpose(1, 2).reshape(B, H, Hq // H * n, D)
    scores = (q @ k.transpose(2, 3)) / math.sqrt(D)
    last = s["lens"].long()[:, None] - n + torch.arange(n, device="cuda")  # [B][n]
    seen = torch.arange(T, device="cuda") <= last[..., None]  # [B][n][T]
    seen = seen[:, None, None].expand(B, H, Hq // H, n, T).reshape(B, H, -1, T)
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = (p @ v).view(B, Hq, n, D).transpose(1, 2)
    s["out"].copy_(o)
    if s["weights"] is None:
        return (s["out"],)
    s["weights"] += p.sum(2)
    return s["out"], s["weights"]


def _evict(s):
    case = s["case"]
    keep, page, D = case["keep"], case["page"], case["dim"]
    w, pos = s["weights"], s["pos"].long()
    B, H, T = w.shape
    slots = torch.arange(T, device="cuda")
    lens = s["lens"].long()
    valid = (slots < lens[:, None])[:, None].expand(B, H, T)
    newest = torch.where(valid, pos, -1).amax(-1, keepdim=True)
    late = valid & (pos > newest - case["recent"])
    # recent tokens first, then by weight, the lower slot first among equals; free slots last
    key = torch.where(late, math.inf, torch.where(valid, w, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(valid).scatter(2, order[..., :keep], True) & valid
    left = torch.minimum(lens, torch.full_like(lens, keep))
    front = (slots < left[:, None])[:, None]
    # the i-th evicted slot in front takes the i-th kept token behind it
    hole, fill = front & ~kept, kept & ~front
    fill_at = torch.full((B, H, T + 1), 0, device="cuda").scatter(
        2, torch.where(fill, fill.cumsum(-1) - 1, T), slots.expand(B, H, T))
    src = torch.where(hole, torch.gather(fill_at, 2, (hole.cumsum(-1) - 1).clamp(min=0)), slots)
    src = torch.where(front, src, slots)[..., :keep]
    at = torch.gather(s["table"].long()[:, None].expand(B, H, -1), 2, src // page)
    to = s["table"].long()[:, None, torch.arange(keep, device="cuda") // page].expand(B, H, keep)
    h = torch.arange(H, device="cuda")[:, None].expand(B, H, keep)
    here, there = src % page, (slots[:keep] % page).expand(B, H, keep)
    s["k_codes"][to, h, there] = s["k_codes"][at, h, here]
    s["scales"][to, h, there] = s["scales"][at, h, here]
    blocks = s["v_codes"].unflatten(-1, (16, D // 64, 4, 2))
    blocks[to, h, there // 4, :, :, there % 4] = blocks[at, h, here // 4, :, :, here % 4]
    s["weights_out"][..., :keep] = torch.where(front[..., :keep], torch.gather(w, 2, src), 0.0)
    s["pos_out"][..., :keep] = torch.where(front[..., :keep], torch.gather(s["pos"], 2, src), 0)
    s["lens_out"].copy_(left)
    return _evict_outputs(s)


def _evict_outputs(s):
    # codes are moved, not computed: they are returned as the bytes they are
    return (s["lens_out"], s["weights_out"], s["pos_out"], s["k_codes"], s["v_codes"],
            s["scales"])


# ------------------------------------------------------------------------------ the least


def work(case):
    size = 2 if case.get("dtype", "f16") == "f16" else 4
    if case["op"] == "linear":
        T, M, K = case["tokens"], case["rows"], case["cols"]
        return {"bytes": T * K * size + M * K + 4 * M + T * M * size
                + (M * size if case["bias"] else 0), "flops": 2 * T * M * K}
    H, D = case["kv_heads"], case["dim"]
    token = H * (D + 8)  # a cached token's codes and scales, K and V
    if case["op"] == "append":
        n = case["batch"] * case["tokens"]
        # the vectors are read, their codes written, and read again for the values written out
        return {"bytes": n * (2 * 2 * H * D * size + 2 * token), "flops": n * H * D * 2 * 6}
    if case["op"] == "attend":
        n, Hq, lens = case["queries"], case["heads"], _lengths(case["batch"], case["context"])
        pairs = sum(max(0, L - n + i + 1) for L in lens for i in range(n)) * Hq
        return {"bytes": sum(lens) * (token + (8 * H if case["weights"] else 0))
                + 2 * case["batch"] * n * Hq * D * size, "flops": 4 * pairs * D}
    rows, L, keep = case["batch"] * H, case["length"], min(case["keep"], case["length"])
    # weights and positions are read once; a kept share of the tail moves: read and written
    moved = (L - keep) * keep / L
    return {"bytes": rows * (8 * L + 8 * keep + 2 * moved * (D + 8)), "flops": rows * L * 8}


# ------------------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x = s["x"].double()
        step = x.abs().max(dim=1).values / 127
        code = (x / torch.where(step > 0, step, torch.ones_like(step)).unsqueeze(1)).round()
        y = code @ s["w"].double().T
        y *= step.unsqueeze(1)
        y *= s["w_scale"].double()
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "append":
        got = []
        for x in (s["k"], s["v"]):
            x = x.double()
            low, high = x.min(dim=-1, keepdim=True).values, x.max(dim=-1, keepdim=True).values
            step, low = ((high - low) / 15).half().double(), low.half().double()
            code = ((x - low) / step).nan_to_num(0, 0, 0).round().clamp(0, 15)
            got.append(low + step * code)
        return tuple(got)
    if case["op"] == "evict":
        return None  # moved bytes and chosen tokens: nothing is computed in floating point
    B, n, Hq, D = s["q"].shape
    H, page = case["kv_heads"], case["page"]
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device="cuda")
    weights = None if s["weights"] is None else s["weights"].double()
    channel = torch.arange(D, device="cuda")
    byte = channel % 64 // 4 * (D // 8) + channel // 64 * 8 + channel % 4 // 2
    for b in range(B):
        L = int(s["lens"][b])
        slot = torch.arange(L, device="cuda")
        pages, line = s["table"][b].long()[slot // page], slot % page
        for h in range(H):
            m = s["scales"][pages, h, line].double()
            c = s["k_codes"][pages, h, line][:, channel // 2].int() >> (channel % 2 * 4) & 15
            key = m[:, 1:2] + m[:, 0:1] * c.double()
            c = s["v_codes"][pages, h, line // 4].gather(
                1, byte + (line % 4 * 2).unsqueeze(1)).int() >> (channel % 2 * 4) & 15
            value = m[:, 3:4] + m[:, 2:3] * c.double()
            for g in range(h * (Hq // H), (h + 1) * (Hq // H)):
                z = s["q"][b, :, g].double() @ key.T / math.sqrt(D)
                z[slot > (L - n + torch.arange(n, device="cuda")).unsqueeze(1)] = -math.inf
                p = torch.softmax(z, dim=1).nan_to_num(0.0)
                out[b, :, g] = p @ value
                if weights is not None:
                    weights[b, h, :L] += p.sum(0)
    return (out,) if weights is None else (out, weights)
