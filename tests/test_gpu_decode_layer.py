"""The low-bit operators together, as examples/decode_layer.py uses them: each stage against its
float64 definition on the stage's own inputs, through a prompt, evictions and a captured step."""

import importlib.util
import os
import sys

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402
from test_gpu_int import tolerance  # noqa: E402
from test_gpu_kv import bound  # noqa: E402

SPEC = importlib.util.spec_from_file_location(
    "decode_layer", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                 "examples", "decode_layer.py"))
decode_layer = importlib.util.module_from_spec(SPEC)
SPEC.loader.exec_module(decode_layer)


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def host(cache):
    """A host copy of a cache."""
    B, H, page, D = cache.batch, cache.heads, cache.page_tokens, cache.head_dim
    c = lb.Cache(cache.k_codes.shape[0], H, page, D, cache.page_table.cpu().numpy(),
                 cache.lens.cpu().numpy())
    c.k, c.v, c.s = (t.cpu().numpy() for t in (cache.k_codes, cache.v_codes, cache.scales))
    return c


def block(**more):
    return decode_layer.AttentionBlock(2, hidden=256, heads=4, kv_heads=2, head_dim=64, keep=40,
                                       recent=8, longest_prompt=70, page_tokens=16, **more)


def test_prompt():
    say("decode_layer prompt")
    b = block()
    kept = []
    evict = bcq.bcq_kv_evict

    def before_eviction(cache, *args, **kw):
        kept.append(host(cache))
        evict(cache, *args, **kw)

    x = torch.randn((2, 70, 256), device="cuda").half()
    mp = pytest.MonkeyPatch()
    mp.setattr(bcq, "bcq_kv_evict", before_eviction)
    try:
        out = b.prompt(x)
    finally:
        mp.undo()
    cache = kept[0]
    assert cache.lens.tolist() == [70, 70] and b.cache.lens.tolist() == [40, 40]
    w = [(c.cpu().numpy(), s.cpu().numpy()) for c, s in b.codes]
    rows = x.cpu().numpy().reshape(140, 256)
    qkv = lb.product(*lb.quantize_rows(rows), *w[0], None)
    got = torch.empty((140, qkv.shape[1]), dtype=torch.float16, device="cuda")
    bcq.bcq_int_linear(x.view(140, 256), *b.codes[0], got)
    assert (np.abs(got.cpu().numpy() - qkv) <= tolerance(qkv, None, "f16")).all()
    q = b.split(got)[0]
    context = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    b2 = block()
    b2.cache.lens.fill_(70)
    bcq.bcq_kv_append(b2.cache, *b.split(got)[1:])
    assert np.array_equal(host(b2.cache).k, cache.k) and np.array_equal(host(b2.cache).v, cache.v)
    bcq.bcq_kv_attend(b2.cache, q, context)
    ref, _, bd, _ = lb.attend(cache, q.cpu().numpy(), np.float32(0.125))
    assert (np.abs(context.cpu().numpy() - ref) <= bound(ref, bd, 64, 70, "f16")).all()
    y = lb.product(*lb.quantize_rows(context.cpu().numpy().reshape(140, 256)), *w[1], None)
    assert (np.abs(out.cpu().numpy().reshape(140, 256) - y) <= tolerance(y, None, "f16")).all()


def test_steps():
    say("decode_layer steps")
    b, other = block(), block()
    x = torch.randn((2, 30, 256), device="cuda").half()
    b.prompt(x)
    other.prompt(x)
    token, out = x[:, 0].contiguous(), torch.empty((2, 256), dtype=torch.float16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, context = b.step(token, out, 2)
    want = torch.empty_like(out)
    for i in range(25):
        token.copy_(torch.randn((2, 256), device="cuda"))
        before = host(b.cache)
        graph.replay()
        other.step(token, want, 2)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert b.cache.lens.tolist() == [min(31 + i, 40)] * 2
        if i < 10:  # nothing is evicted yet, so the cache is what was attended
            after = host(b.cache)
            assert after.lens.tolist() == [before.lens[0] + 1] * 2
            ref, _, bd, _ = lb.attend(after, q.cpu().numpy(), np.float32(0.125))
            err = np.abs(context.cpu().numpy() - ref)
            assert (err <= bound(ref, bd, 64, 40, "f16")).all(), i
    newest = b.pos[..., :40].sort(-1).values[..., -8:]
    assert (newest == torch.arange(47, 55, device="cuda")).all()
