"""The operators of a packed serving step, as they are measured: requests of unlike lengths, prompts
and single tokens together, as one list of tokens without padding.

* ``norm``: residual addition, root-mean-square norm and an output in 8 bits with a scale a token,
  as the 8-bit products read it (or in the call's type, as the planes' products do);
* ``reserve``: pages of the 4-bit cache given out and taken back, page tables, starts, slots and
  positions of the step's tokens from the requests' lengths;
* ``append``: the step's keys and values quantized into those slots, and read back;
* ``attend``: causal attention of all the step's tokens over the cache, whose sequences may share
  a long prefix that is read once for all.

``run(state)`` is one pass: the plain form of torch operations in 32 bits where ``own`` is False,
the library's entry points where it is True.  Both take the same state and return the same
outputs.  ``exact(case, seed)`` is the definition in 64 bits.

Formats (bytes as the library defines them):

* 8-bit rows: code = rint(y / s), s = max|y| / 127 for each row; value = s * code.
* 4-bit vectors: one fp16 scale and one fp16 zero for each (token, head, K or V) vector of D
  channels; zero = min, scale = (max - min) / 15, code = clamp(rint((x - zero) / scale), 0, 15);
  value = zero + scale * code.
* Pages of ``page`` tokens: K codes [pages][heads][page][D/2], two channels a byte, the even one
  in the low half; V codes [pages][heads][page/4][16][D/64][4][2]: blocks of four tokens, in a
  block byte (r, h, t, c) holds channels 64h + 4r + 2c and + 1 of its token t; scales
  [pages][heads][page][4] = (K scale, K zero, V scale, V zero).
* A slot is page * page_tokens + the token's place in the page.
"""

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # one request's token between two planes' products: latency
        {"name": "norm 1x4096 f16", "op": "norm", "dtype": "f16", "tokens": 1, "cols": 4096,
         "out": "values"},
        # odd sizes in both directions, single precision, into 8 bits
        {"name": "norm 515x1001 f32", "op": "norm", "dtype": "f32", "tokens": 515, "cols": 1001,
         "out": "codes"},
        # prompts of 4096 tokens on their way into an 8-bit product
        {"name": "norm 4096x4096 f16", "op": "norm", "dtype": "f16", "tokens": 4096,
         "cols": 4096, "out": "codes"},
        # a decode step of 64 requests: one in 64 needs a new page
        {"name": "reserve 64 decodes", "op": "reserve", "batch": 64, "page": 64, "prompts": 0,
         "longest": 1, "context": 3000, "shared": 0},
        # a step that takes in new prompts where finished requests have left, behind shared pages
        {"name": "reserve 200 with 24 prompts", "op": "reserve", "batch": 200, "page": 32,
         "prompts": 24, "longest": 1500, "context": 4000, "shared": 1024},
        # keys and values of a chunk of a prompt and of 63 single tokens
        {"name": "append 63x1 1x1000 f16", "op": "append", "dtype": "f16", "batch": 64,
         "prompts": 1, "longest": 1000, "drafts": 1, "kv_heads": 8, "dim": 128, "page": 64,
         "context": 1500},
        # prompts of odd lengths, single precision, small pages
        {"name": "append 9 prompts f32", "op": "append", "dtype": "f32", "batch": 9,
         "prompts": 9, "longest": 1501, "drafts": 1, "kv_heads": 8, "dim": 64, "page": 16,
         "context": 0},
        # a few requests behind a common instruction: latency
        {"name": "attend 4x1 shared 1024 f16", "op": "attend", "dtype": "f16", "batch": 4,
         "prompts": 0, "longest": 1, "drafts": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "context": 300, "shared": 1024},
        # a serving batch behind one long document
        {"name": "attend 64x1 shared 16384 f16", "op": "attend", "dtype": "f16", "batch": 64,
         "prompts": 0, "longest": 1, "drafts": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "context": 1000, "shared": 16384},
        # drafted tokens of a dozen requests, every head with its own keys, single precision
        {"name": "attend 12x5 shared 992 f32", "op": "attend", "dtype": "f32", "batch": 12,
         "prompts": 0, "longest": 5, "drafts": 5, "heads": 16, "kv_heads": 16, "dim": 64,
         "page": 16, "context": 701, "shared": 992},
        # a chunk of one long prompt among the single tokens of 31 requests
        {"name": "attend 31x1 1x1024 f16", "op": "attend", "dtype": "f16", "batch": 32,
         "prompts": 1, "longest": 1024, "drafts": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "context": 6000, "shared": 0},
        # whole prompts of unlike lengths: bound by the matrix cores
        {"name": "attend 6 prompts f16", "op": "attend", "dtype": "f16", "batch": 6,
         "prompts": 6, "longest": 4001, "drafts": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 128, "context": 0, "shared": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (16, 16), (28, 4), (8, 1), (12, 12), (64, 8), (40, 8)]


def draw(rng):
    op = rng.choice(["norm", "norm", "reserve", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["f16", "f16", "f32"])
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    if op == "norm":
        cols = _log(rng, 64, 14336)
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 4096 * 4096 // cols),
                "cols": cols, "out": rng.choice(["values", "codes"])}
    if op == "reserve":
        batch = _log(rng, 1, 256)
        prompts = rng.choice([0, 1, _log(rng, 1, 24)])
        longest = _log(rng, 2, 1500) if prompts else 1
        return {"op": op, "batch": max(batch, prompts), "page": page, "prompts": prompts,
                "longest": longest, "context": _log(rng, 10, 4000),
                "shared": rng.choice([0, page * rng.randint(1, 16)])}
    batch = _log(rng, 1, 64)
    prompts = rng.choice([0, 0, 1, _log(rng, 1, 6)])
    batch = max(batch, prompts)
    drafts = rng.choice([1, 1, 1, 2, 5])
    if op == "append":
        return {"op": op, "dtype": dtype, "batch": batch, "prompts": prompts,
                "longest": _log(rng, 2, 1500) if prompts else drafts, "drafts": drafts,
                "kv_heads": rng.choice([1, 4, 8, 16]), "dim": dim, "page": page,
                "context": _log(rng, 1, 2000)}
    heads, kv_heads = rng.choice(HEADS)
    context = _log(rng, 1, min(8000, 65536 * 8 // (batch * max(8, kv_heads))))
    shared = rng.choice([0, 0, page * _log(rng, 1, 16384 // page)]) if batch > 1 else 0
    most = 6 * 3000 * 1500 * 32 * 128  # products, of all the prompts
    longest = drafts
    if prompts:
        longest = _log(rng, 2, 3000)
        while longest > 2 and prompts * longest * (context + shared + longest) * heads * dim > most:
            longest = longest * 3 // 4
    return {"op": op, "dtype": dtype, "batch": batch, "prompts": prompts, "longest": longest,
            "drafts": drafts, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "context": context, "shared": shared}


def _step(case):
    """(cached tokens before the step, behind the shared ones; new tokens) of every sequence: prompts
    spread among the sequences, from the longest down to about half of it, over contexts likewise."""
    B, P = case["batch"], case["prompts"]
    context, new = [], []
    at = {(i * B) // P: i for i in range(P)} if P else {}
    for b in range(B):
        c = case["context"]
        context.append(c - b * (c // 2) // B)
        i = at.get(b)
        longest = case["longest"]
        new.append(case.get("drafts", 1) if i is None else longest - i * (longest // 2) // P)
    return context, new


# ------------------------------------------------------------------------------ inputs


def _pad(n, m):
    return (n + m - 1) // m * m


def _pages(n, page):
    return (n + page - 1) // page


def _starts(new):
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    return at


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _cache(case, lens, g):
    """Random codes, scales and zeros in scattered pages; the first pages of all are the same."""
    page, H, D, shared = case["page"], case["kv_heads"], case["dim"], case.get("shared", 0)
    B, ahead = len(lens), shared // page
    width = max(_pages(n, page) for n in lens)
    pages = ahead + B * (width - ahead)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.cat([order[:ahead].expand(B, ahead), order[ahead:].view(B, width - ahead)], 1)

    def codes(shape):
        # nearly as the codes of a bell curve lie: the sum of four numbers of 0 to 3 and one more
        b = torch.randint(0, 256, (2,) + shape, generator=g, device="cuda", dtype=torch.uint8)
        parts = [(b[i] >> s & 3) + (b[i] >> (s + 2) & 3) for i in (0, 1) for s in (0, 4)]
        low, high = parts[0] + parts[1], parts[2] + parts[3]
        return low | high << 4

    n = pages * H * page
    f = torch.rand((n, 4), generator=g, device="cuda")
    # 15 steps of 0.3 to 0.4 about zero: a spread of about 1
    f[:, 0::2] = 0.3 + 0.1 * f[:, 0::2]
    f[:, 1::2] = -2.4 + 0.3 * f[:, 1::2]
    return {
        "k_codes": codes((pages, H, page, D // 2)),
        "v_codes": codes((pages, H, page // 4, 2 * D)),
        "scales": f.half().view(pages, H, page, 4),
        "table": table.contiguous(),
        "lens": _ints(lens),
    }


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    state = {"case": dict(case)}
    dt = DTYPES[case.get("dtype", "f16")]
    if case["op"] == "norm":
        T, K = case["tokens"], case["cols"]
        # a residual stream with a hundredth of its channels twenty times larger
        r = torch.randn((T, _pad(K, 16)), generator=g, device="cuda")
        r[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 20
        x = torch.randn((T, _pad(K, 16)), generator=g, device="cuda")
        gamma = 1 + 0.2 * torch.randn(K, generator=g, device="cuda")
        state.update(x=x.to(dt)[:, :K], residual=r.to(dt)[:, :K], gamma=gamma.to(dt),
                     h=torch.empty_like(x, dtype=dt)[:, :K],
                     y=torch.empty((T, _pad(K, 16)), dtype=dt, device="cuda")[:, :K])
        if case["out"] == "codes":
            state.update(codes=torch.zeros((T, _pad(K, 16)), dtype=torch.int8,
                                           device="cuda")[:, :K],
                         scales=torch.empty(T, device="cuda"))
        return state
    if case["op"] == "reserve":
        return _prepare_reserve(case, state, g, seed)
    before, new = _step(case)
    shared, T = case.get("shared", 0), sum(new)
    state.update(_cache(case, [shared + c + n for c, n in zip(before, new)], g),
                 starts=_ints(_starts(new)), max_n=max(new), new=new)
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        # keys and values lie behind the queries in one projection's output
        qkv = torch.randn((T, 4 * H, D), generator=g, device="cuda").to(dt)
        b = torch.repeat_interleave(torch.arange(len(new), device="cuda"), _ints(new).long())
        slot = torch.arange(T, device="cuda") - state["starts"].long()[b] + _ints(before).long()[b]
        at = state["table"].long()[b, slot // page]
        state.update(k=qkv[:, 2 * H:3 * H], v=qkv[:, 3 * H:], slots=at * page + slot % page,
                     k_out=torch.empty((T, H, D), dtype=dt, device="cuda"),
                     v_out=torch.empty((T, H, D), dtype=dt, device="cuda"))
        return state
    q = torch.randn((T, case["heads"], D), generator=g, device="cuda").to(dt)
    state.update(q=q, out=torch.zeros_like(q))
    return state


def _prepare_reserve(case, state, g, seed):
    """Sequences of a running server: pages in no order, a stack of the free ones.  Where prompts
    start, another request has just ended (or nothing was there)."""
    rng = random.Random(seed)
    page, ahead = case["page"], case["shared"] // case["page"]
    before, new = _step(case)
    before = [max(0, c - rng.randrange(page)) for c in before]
    B, P = case["batch"], case["prompts"]
    begins = {(i * B) // P for i in range(P)}
    release = [1 if b in begins else 0 for b in range(B)]
    if not P:
        release = [0] * B
    own_pages = [_pages(c, page) for c in before]
    width = ahead + _pages(case["context"] + case["longest"], page) + 1
    spare = sum(_pages(n, page) + 1 for n in new)
    pages = ahead + B * _pages(case["context"], page) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = ahead
    ids = order.cpu()
    for b in range(B):
        table[b, :ahead] = ids[:ahead]
        table[b, ahead:ahead + own_pages[b]] = ids[at:at + own_pages[b]]
        at += own_pages[b]
    free = torch.full((pages,), -1, dtype=torch.int32)
    free[:spare] = ids[at:at + spare]
    T = sum(new)
    zeros = lambda shape, dt: torch.zeros(shape, dtype=dt, device="cuda")  # noqa: E731
    state.update(
        # the tables need no more of a cache than its pages' number: one head of 64 channels
        k_codes=zeros((pages, 1, page, 32), torch.uint8),
        v_codes=zeros((pages, 1, page // 4, 128), torch.uint8),
        scales=zeros((pages, 1, page, 4), torch.float16),
        table=table.cuda(), lens=_ints([ahead * page + c for c in before]),
        new=_ints(new), release=_ints(release), free=free.cuda(), count=_ints([spare]),
        starts=zeros(B + 1, torch.int32), slots=zeros(T, torch.int64),
        positions=zeros(T, torch.int32), lens_out=zeros(B, torch.int32),
        table_out=zeros((B, width), torch.int32), free_out=zeros(pages, torch.int32),
        count_out=zeros(1, torch.int32))
    return state


# ------------------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "reserve": _own_reserve, "append": _own_append,
                "attend": _own_attend}[op](state)
    return {"norm": _norm, "reserve": _reserve, "append": _append, "attend": _attend}[op](state)


def _handle(bcq, s):
    """The cache's handle, made once, as a program keeps it with its cache."""
    h = s.get("handle")
    if h is None:
        h = s["handle"] = bcq.KVCache(s["k_codes"], s["v_codes"], s["scales"], s["table"],
                                      s["lens"])
    return h


def _own_norm(s):
    import binary_coded_precision_amd as bcq

    if s["case"]["out"] == "values":
        bcq.bcq_rms_norm(s["x"], s["gamma"], EPS, residual=s["residual"], H=s["h"], Y=s["y"])
        return s["h"], s["y"]
    bcq.bcq_rms_norm(s["x"], s["gamma"], EPS, residual=s["residual"], H=s["h"], codes=s["codes"],
                     scales=s["scales"])
    return _values(s)


def _own_reserve(s):
    import binary_coded_precision_amd as bcq

    h = _handle(bcq, s)
    if "workspace" not in s:
        s["workspace"] = bcq.new_kv_reserve_workspace(h)
    bcq.bcq_kv_reserve(h, s["new"], s["free"], s["count"], s["starts"], s["slots"],
                       s["positions"], release=s["release"],
                       shared_pages=s["case"]["shared"] // s["case"]["page"],
                       lens_out=s["lens_out"], page_table_out=s["table_out"],
                       free_pages_out=s["free_out"], free_count_out=s["count_out"],
                       workspace=s["workspace"])
    return _reserve_outputs(s)


def _own_append(s):
    import binary_coded_precision_amd as bcq

    h = _handle(bcq, s)
    bcq.bcq_kv_append_slots(h, s["k"], s["v"], s["slots"])
    bcq.bcq_kv_read_slots(h, s["k_out"], s["v_out"], s["slots"])
    return s["k_out"], s["v_out"]


def _own_attend(s):
    import binary_coded_precision_amd as bcq

    h = _handle(bcq, s)
    ahead = s["case"]["shared"] // s["case"]["page"]
    if "workspace" not in s:
        s["workspace"] = bcq.new_kv_packed_workspace(h, *s["q"].shape[:2], s["max_n"],
                                                     shared_pages=ahead)
    bcq.bcq_kv_attend_packed(h, s["q"], s["out"], s["starts"], s["max_n"], shared_pages=ahead,
                             workspace=s["workspace"])
    return s["out"]


# ------------------------------------------------------------------------------ plain forms


def _values(s):
    """The values that the codes stand for, in the call's type."""
    return s["h"], torch.mul(s["codes"], s["scales"].unsqueeze(1), out=s["y"])


def _norm(s):
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    s["h"].copy_(h)
    h = h.float()
    # the mean in 64 bits: the codes are rounded from what it scales
    mean = (h.double() * h.double()).mean(1, keepdim=True)
    y = h * (1 / torch.sqrt(mean + EPS)).float() * s["gamma"].float()
    if s["case"]["out"] == "values":
        s["y"].copy_(y)
        return s["h"], s["y"]
    scale = y.abs().amax(1) * (1 / 127)
    s["scales"].copy_(scale)
    s["codes"].copy_(torch.round(y / torch.where(scale > 0, scale, 1.0).unsqueeze(1)))
    return _values(s)


def _reserve_outputs(s):
    return (s["starts"], s["slots"], s["positions"], s["lens_out"], s["table_out"],
            s["free_out"], s["count_out"])


def _reserve(s):
    page, ahead = s["case"]["page"], s["case"]["shared"] // s["case"]["page"]
    table, free, T = s["table"].long(), s["free"].long(), s["slots"].shape[0]
    B, width = table.shape
    gone, lens, want = s["release"] != 0, s["lens"].long(), s["new"].long().clamp(min=0)
    # pages that come back go on top of the stack, in the tables' order
    back = torch.where(gone, (_pages(lens, page) - ahead).clamp(min=0), 0)
    count = s["count"].long()
    entry = torch.arange(width, device="cuda")
    off = (count + back.cumsum(0) - back)[:, None] + entry - ahead
    given = (entry >= ahead) & (entry < ahead + back[:, None])
    stack = torch.cat([free, free.new_zeros(1)])
    stack = stack.scatter(0, torch.where(given, off, len(free)).flatten(), table.flatten())
    top = count + back.sum()
    # in the sequences' order, all pages that a request needs or none
    lens = torch.where(gone, ahead * page, lens)
    first = _pages(lens, page).clamp(min=ahead)
    fits = lens + want <= width * page
    want = torch.where(fits, want, 0)
    need = _pages(lens + want, page).clamp(min=ahead) - first
    granted = fits & (want.cumsum(0) <= T) & ((need == 0) | (need.cumsum(0) <= top))
    base = need.cumsum(0) - need
    n = torch.where(granted, want, 0)
    need = torch.where(granted, need, 0)
    new = (entry >= first[:, None]) & (entry < (first + need)[:, None])
    take = (top - 1 - base)[:, None] - (entry - first[:, None])
    table = torch.where(new, stack[torch.where(new, take, 0)], table)
    last = lens + n
    s["table_out"].copy_(torch.where(entry < _pages(last, page)[:, None], table,
                                     s["table_out"].long()))
    s["lens_out"].copy_(last)
    left = top - need.sum()
    s["count_out"].copy_(left)
    s["free_out"].copy_(torch.where(torch.arange(len(free), device="cuda") < left, stack[:-1],
                                    s["free_out"].long()))
    ends = n.cumsum(0)
    s["starts"][1:] = ends
    # a token's sequence, position and slot; -1 past the last token
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    at = lens[b] + t - (ends - n)[b]
    there = t < ends[-1]
    s["positions"].copy_(torch.where(there, at, -1))
    page_of = table[b, torch.where(there, at // page, 0)]
    s["slots"].copy_(torch.where(there, page_of * page + at % page, -1))
    return _reserve_outputs(s)


def _four_bits(x):
    """(codes, scale, zero) of vectors along the last dimension, as the library's format says."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale, zero = ((hi - lo) * (1 / 15)).half(), lo.half()
    s = scale.float()
    q = torch.where(s > 0, (x - zero.float()) / torch.where(s > 0, s, 1.0), 0.0)
    return torch.round(q).clamp(0, 15).to(torch.uint8), scale, zero


def _nibbles(b):
    """Bytes [..., n] as the 2n codes they hold."""
    return torch.stack([b & 15, b >> 4], -1).flatten(-2).float()


def _append(s):
    page, D = s["case"]["page"], s["case"]["dim"]
    at, line = s["slots"] // page, s["slots"] % page
    ck, sk, zk = _four_bits(s["k"])
    cv, sv, zv = _four_bits(s["v"])
    # after the two indexes, the token's own dimensions: [T][H][...]
    s["k_codes"][at, :, line] = ck[..., 0::2] | ck[..., 1::2] << 4
    v = cv.unflatten(-1, (D // 64, 16, 2, 2))
    v = (v[..., 0] | v[..., 1] << 4).transpose(-3, -2)  # [T][H][r][h][c]
    blocks = s["v_codes"].unflatten(-1, (16, D // 64, 4, 2))
    blocks[at, :, line // 4, :, :, line % 4] = v
    s["scales"][at, :, line] = torch.cat([sk, zk, sv, zv], -1)
    # and read back as the values that they stand for
    c, m = _nibbles(s["k_codes"][at, :, line]), s["scales"][at, :, line].float()
    s["k_out"].copy_(c * m[..., 0:1] + m[..., 1:2])
    c = _nibbles(blocks[at, :, line // 4, :, :, line % 4].transpose(-3, -2)).flatten(-3)
    s["v_out"].copy_(c * m[..., 2:3] + m[..., 3:4])
    return s["k_out"], s["v_out"]


def _unpack(s, pages):
    """Keys and values of the pages in 32 bits, [...][heads][page][D]."""
    sc = s["scales"][pages].float()
    k = _nibbles(s["k_codes"][pages]) * sc[..., 0:1] + sc[..., 1:2]
    D = k.shape[-1]
    v = s["v_codes"][pages].unflatten(-1, (16, D // 64, 4, 2))  # [...][T/4][r][h][t][c]
    v = v.movedim(-2, -4).transpose(-3, -2)  # [...][T/4][t][h][r][c]
    v = _nibbles(v).flatten(-3).flatten(-3, -2)  # [...][T][D]
    return k, v * sc[..., 2:3] + sc[..., 3:4]


def _attend_padded(s, seqs, n):
    """Sequences of up to n new tokens, as a batch padded to the longest; results in place."""
    seqs = _ints(seqs, torch.int64)
    length, start = s["lens"].long()[seqs], s["starts"].long()[seqs]
    mine = s["starts"].long()[seqs + 1] - start
    i = torch.arange(n, device="cuda")
    there = i < mine[:, None]  # [B][n]
    token = torch.where(there, start[:, None] + i, start[:, None])
    q = s["q"][token].float()  # [B][n][Hq][D]
    B, _, Hq, D = q.shape
    k, v = (t.transpose(1, 2).flatten(2, 3) for t in _unpack(s, s["table"].long()[seqs]))
    H, T = k.shape[1], k.shape[2]
    # rows of a cached head: its queries' heads, all the queries of each
    q = q.transpose(1, 2).reshape(B, H, Hq // H * n, D)
    scores = (q @ k.transpose(2, 3)) / math.sqrt(D)
    last = (length - mine)[:, None] + i
    hidden = torch.arange(T, device="cuda") > last[..., None]  # [B][n][T]
    scores.view(B, Hq, n, T).masked_fill_(hidden[:, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    o = (scores @ v) / scores.sum(-1, keepdim=True)
    o = o.view(B, Hq, n, D).transpose(1, 2)
    s["out"][token[there]] = o[there].to(s["out"].dtype)


def _attend(s):
    # single and drafted tokens as one batch, prompts as another
    few = [b for b, n in enumerate(s["new"]) if n <= s["case"]["drafts"]]
    many = [b for b, n in enumerate(s["new"]) if n > s["case"]["drafts"]]
    if few:
        _attend_padded(s, few, s["case"]["drafts"])
    if many:
        _attend_padded(s, many, s["max_n"])
    return s["out"]


# ------------------------------------------------------------------------------ the least


def work(case):
    size = 2 if case.get("dtype", "f16") == "f16" else 4
    if case["op"] == "norm":
        n, codes = case["tokens"] * case["cols"], case["out"] == "codes"
        # codes are written, and read again for the values they stand for
        return {"bytes": n * (4 * size + (2 if codes else 0)) + case["cols"] * size, "flops": 8 * n}
    before, new = _step(case)
    T, page, shared = sum(new), case["page"], case.get("shared", 0)
    if case["op"] == "reserve":
        entries = sum(shared // page + _pages(c + n, page) for c, n in zip(before, new))
        return {"bytes": 12 * T + 8 * entries + 20 * case["batch"], "flops": 10 * T}
    H, D = case["kv_heads"], case["dim"]
    token = H * (D + 8)  # a cached token's codes and scales, K and V
    if case["op"] == "append":
        # the vectors are read, their codes written, and read again for the values written out
        return {"bytes": T * (2 * 2 * H * D * size + 2 * token), "flops": T * H * D * 2 * 6}
    pairs = sum(n * (shared + c) + n * (n + 1) // 2 for c, n in zip(before, new))
    return {"bytes": (shared + sum(before) + T) * token + 2 * T * case["heads"] * D * size,
            "flops": 4 * pairs * case["heads"] * D}


# ------------------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
        rms = h.pow(2).sum(1).div(case["cols"]).add(EPS).sqrt()
        if case["out"] == "values":
            return h, h / rms.unsqueeze(1) * s["gamma"].double()
        # the format defines codes in single precision, from the normed values rounded to it
        y = (h.float() * rms.reciprocal().float().unsqueeze(1)) * s["gamma"].float()
        step = (y.abs().max(dim=1).values * torch.tensor(1 / 127, device="cuda")).unsqueeze(1)
        return h, (y / step).nan_to_num(0).round().double() * step.double()
    if case["op"] == "append":
        got = []
        for x in (s["k"], s["v"]):
            # the format defines scale, zero and codes in single precision
            x = x.float()
            low, high = x.min(dim=-1, keepdim=True).values, x.max(dim=-1, keepdim=True).values
            step = (high - low).mul(torch.tensor(1 / 15, device="cuda")).half()
            code = ((x - low.half().float()) / step.float()).nan_to_num(0, 0, 0)
            got.append(low.half().double() + step.double() * code.round().clamp(0, 15).double())
        return tuple(got)
    if case["op"] == "reserve":
        return None  # whole numbers
    T, Hq, D = s["q"].shape
    H, page = case["kv_heads"], case["page"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    channel = torch.arange(D, device="cuda")
    byte = channel % 64 // 4 * (D // 8) + channel // 64 * 8 + channel % 4 // 2
    at = 0
    for b, n in enumerate(s["new"]):
        L = int(s["lens"][b])
        slot = torch.arange(L, device="cuda")
        pages, line = s["table"][b].long()[slot // page], slot % page
        hidden = slot > (L - n + torch.arange(n, device="cuda")).unsqueeze(1)
        for h in range(H):
            m = s["scales"][pages, h, line].double()
            c = s["k_codes"][pages, h, line][:, channel // 2].int() >> (channel % 2 * 4) & 15
            key = m[:, 1:2] + m[:, 0:1] * c.double()
            c = s["v_codes"][pages, h, line // 4].gather(
                1, byte + (line % 4 * 2).unsqueeze(1)).int() >> (channel % 2 * 4) & 15
            value = m[:, 3:4] + m[:, 2:3] * c.double()
            for g in range(h * (Hq // H), (h + 1) * (Hq // H)):
                z = s["q"][at:at + n, g].double() @ key.T / math.sqrt(D)
                z.masked_fill_(hidden, -math.inf)
                out[at:at + n, g] = torch.softmax(z, dim=1) @ value
        at += n
    return out
