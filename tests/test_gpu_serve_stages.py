"""Packed steps of examples/serve_layers.py, stage by stage: every operator's call is recorded, its
inputs have to be what the stages before it gave, and its outputs what its definition makes of
them.  test_packed_accuracy plants mistakes that the attention's bound has to tell."""

import sys
from types import SimpleNamespace

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_int import tolerance  # noqa: E402
from test_gpu_kv_packed import reference  # noqa: E402
from test_gpu_serve_layers import serve_layers, server, tokens  # noqa: E402
from test_lowbit_accuracy import outputs_hold  # noqa: E402

bcq = serve_layers.bcq


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def down(t):
    return t.detach().cpu().numpy().copy()


@pytest.fixture
def recorded(monkeypatch):
    """The calls made, in their order: names, arguments and their values before and after."""
    calls = []

    def record(name, names):
        fn = getattr(bcq, name)

        def call(*args, **kw):
            given = dict(zip(names, args), **kw)
            if "cache" in given:
                cache = given["cache"]
                given.update(k_codes=cache.k_codes, v_codes=cache.v_codes,
                             cache_scales=cache.scales, table=cache.page_table, lens=cache.lens)
            there = {n: v for n, v in given.items()
                     if isinstance(v, torch.Tensor) and n != "workspace"}
            before = {n: down(v) for n, v in there.items()}
            fn(*args, **kw)
            calls.append(SimpleNamespace(
                name=name, was=SimpleNamespace(**before), args=given,
                now=SimpleNamespace(**{n: down(v) for n, v in there.items()})))

        monkeypatch.setattr(bcq, name, call)

    record("bcq_kv_reserve", ("cache", "new_tokens", "free_pages", "free_count", "starts", "slots",
                              "positions"))
    record("bcq_rms_norm", ("X", "gamma", "eps"))
    record("bcq_int_gemm", ("codes", "scales", "W", "w_scales", "Y"))
    record("bcq_kv_append_slots", ("cache", "K", "V", "slots"))
    record("bcq_kv_attend_packed", ("cache", "Q", "O", "starts", "max_n"))
    record("bcq_int_linear", ("X", "W", "w_scales", "Y"))
    return calls


def same(a, b):
    np.testing.assert_array_equal(a, b)


def host(call, table, lens):
    _, H, page, half = call.was.k_codes.shape
    c = lb.Cache(1, H, page, 2 * half, table, lens)
    c.k, c.v, c.s = (x.copy() for x in (call.was.k_codes, call.was.v_codes,
                                        call.was.cache_scales))
    return c


def check_norm(call, x, residual, gamma):
    assert call.name == "bcq_rms_norm" and call.args["eps"] == serve_layers.EPS
    same(call.was.X, x)
    assert (call.args.get("residual") is None) == (residual is None)
    if residual is not None:
        same(call.was.residual, residual)
    same(call.was.gamma, down(gamma))
    h, _, codes, scales = lb.rms_norm(x, residual, down(gamma), serve_layers.EPS)
    same(call.now.H, h)
    same(call.now.codes, codes)
    same(call.now.scales, scales)
    return h, codes, scales


def check_product(call, codes, scales, weights):
    w, ws = (down(t) for t in weights)
    same(call.was.W, w)
    same(call.was.w_scales, ws)
    want = lb.product(codes, scales, w, ws)
    assert (np.abs(call.now.Y - want) <= tolerance(want, None, "f16")).all()
    return call.now.Y


def check_step(s, calls, x, after):
    """All calls of one step from x to `after`; the step's starts."""
    r = calls.pop(0)
    assert r.name == "bcq_kv_reserve"
    T = len(r.was.slots)
    lens, table, free, count, starts, slots, positions = lb.reserve(
        r.was.lens, r.was.table, r.was.free_pages, int(r.was.free_count[0]), r.was.new_tokens,
        r.was.release, s.shared_pages, s.page, T)
    for got, want in ((r.now.lens, lens), (r.now.table, table), (r.now.starts, starts),
                      (r.now.slots, slots), (r.now.positions, positions)):
        same(got, want)
    same(r.now.free_pages[:count], free[:count])
    added = None
    for layer in s.layers:
        norm, qkv, append, attend, out, norm2, gate_up, last = calls[:8]
        del calls[:8]
        x, codes, scales = check_norm(norm, x, added, layer.norms[0])
        assert (qkv.name, append.name, attend.name, out.name) == (
            "bcq_int_gemm", "bcq_kv_append_slots", "bcq_kv_attend_packed", "bcq_int_linear")
        same(qkv.was.codes, codes)
        y = check_product(qkv, codes, scales, layer.qkv).reshape(T, -1, s.dim)
        # keys and values to the bit, in the slots of the step's tokens and nowhere else
        same(append.was.K, y[:, s.heads:s.heads + s.kv_heads])
        same(append.was.V, y[:, s.heads + s.kv_heads:])
        same(append.was.slots, slots)
        c = host(append, np.arange(s.pages)[None], [0])
        for t in range(starts[-1]):
            for h in range(s.kv_heads):
                c.put(0, h, int(slots[t]), append.was.K[t, h], append.was.V[t, h])
        for got, want in ((append.now.k_codes, c.k), (append.now.v_codes, c.v),
                          (append.now.cache_scales.view(np.uint16), c.s.view(np.uint16))):
            same(got, want)
        assert append.args["cache"] is attend.args["cache"] is layer.cache
        same(attend.was.k_codes, c.k)
        # attention over what each request has cached, with lengths and tables of the host
        same(attend.was.Q, y[:, :s.heads])
        same(attend.was.starts, starts)
        ref = reference(host(attend, table, lens), attend.was.Q, starts,
                        float(np.float32(s.dim ** -0.5)))
        assert outputs_hold(attend.now.O[:starts[-1]], ref[:starts[-1]])
        for a, b in zip(starts[:-1], starts[1:]):
            assert a == b or outputs_hold(attend.now.O[a:b], ref[a:b])
        same(attend.now.O[starts[-1]:], attend.was.O[starts[-1]:])
        same(out.was.X, attend.now.O.reshape(T, -1))
        sub = check_product(out, *lb.quantize_rows(out.was.X), layer.out)
        x, codes, scales = check_norm(norm2, x, sub, layer.norms[1])
        assert (gate_up.name, last.name) == ("bcq_int_gemm", "bcq_int_linear")
        same(gate_up.was.codes, codes)
        gate, up = np.split(check_product(gate_up, codes, scales, layer.gate_up)
                            .astype(np.float64), 2, axis=1)
        # the sigmoid's product and the product with `up`, each rounded to fp16
        want = gate / (1 + np.exp(-gate)) * up
        near = 2.01 * 2.0**-11 * np.abs(want) + 2.0**-24 * (1 + np.abs(up))
        assert (np.abs(last.was.X - want) <= near).all()
        added = check_product(last, *lb.quantize_rows(last.was.X), layer.down)
    same(after, (x.astype(np.float32) + added.astype(np.float32)).astype(np.float16))
    assert not calls
    return starts


def step(s, calls, x, new, release=None, T=None):
    t = serve_layers.Step(s, T or len(x), max(new))
    t.x[:len(x)] = x
    t.new.copy_(torch.tensor(new))
    if release is not None:
        t.release.copy_(torch.tensor(release))
    before = down(t.x)
    s.run(t)
    return check_step(s, calls, before, down(t.x)).tolist()


def test_prompts_single_tokens_and_requests_that_end(recorded):
    """Behind a common prompt, and a step that there are not pages enough for."""
    say("serve_layers stages behind a common prompt")
    s = server(4, pages=24)
    x = tokens(48, 0)
    after = s.common(x)
    s.shared_pages = 0  # as it was in that step
    assert check_step(s, recorded, down(x), down(after)).tolist() == [0, 48, 48, 48, 48]
    s.shared_pages = 3
    assert step(s, recorded, tokens(63, 1), [5, 40, 1, 17], T=70) == [0, 5, 45, 46, 63]
    assert step(s, recorded, tokens(4, 2), [1] * 4) == [0, 1, 2, 3, 4]
    assert step(s, recorded, tokens(64, 3), [1, 60, 0, 3], release=[0, 1, 1, 0]) == \
        [0, 1, 61, 61, 64]
    assert s.lens.tolist() == [55, 108, 48, 69]
    assert step(s, recorded, tokens(141, 4), [1, 1, 139, 0]) == [0, 1, 2, 141, 141]
    # one page too few for the last
    left = int(s.count) * s.page
    assert step(s, recorded, tokens(left + 40, 5), [1, 1, 1, left + 37]) == [0, 1, 2, 3, 3]


def test_requests_with_nothing_in_common(recorded):
    say("serve_layers stages alone")
    s = server(3)
    assert step(s, recorded, tokens(97, 6), [32, 1, 64]) == [0, 32, 33, 97]
    assert step(s, recorded, tokens(11, 7), [0, 9, 2]) == [0, 0, 9, 11]
