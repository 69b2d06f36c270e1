"""Decoder layers serving requests of unlike lengths in packed steps, behind a common prompt.

A step's tokens, prompts of new requests and single tokens of running ones, lie one behind the
other without padding.  bcq_kv_reserve takes back the pages of requests that ended and gives pages
and slots to the step's tokens, once for all layers; then every layer norms its rows into 8 bits
(bcq_rms_norm), multiplies them (bcq_int_gemm), appends keys and values by slot
(bcq_kv_append_slots) and attends over what each request has cached (bcq_kv_attend_packed), the
pages of the common prompt read once for all requests that bring few tokens.  A step of single
tokens is captured once in a graph: lengths, starts and tables are on the device.

    python examples/serve_layers.py [--batch 32] [--layers 2] [--common 1024] [--steps 100]
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import binary_coded_precision_amd as bcq  # noqa: E402

EPS = 1e-5


class Layer:
    """One decoder layer: random weights in 8 bits, and its keys and values in the server's pages."""

    def __init__(self, s, g):
        h, q, kv, f = s.hidden, s.heads * s.dim, s.kv_heads * s.dim, s.inner
        self.qkv, self.out, self.gate_up, self.down = (
            bcq.bcq_int_quantize(torch.randn(shape, generator=g, device="cuda")
                                 .mul_(shape[1] ** -0.5).half())
            for shape in ((q + 2 * kv, h), (h, q), (2 * f, h), (h, f)))
        self.norms = torch.ones((2, h), dtype=torch.float16, device="cuda")
        pages = lambda *shape: torch.zeros(  # noqa: E731
            (s.pages, s.kv_heads, *shape), dtype=torch.uint8, device="cuda")
        self.cache = bcq.KVCache(
            pages(s.page, s.dim // 2), pages(s.page // 4, 2 * s.dim),
            torch.zeros((s.pages, s.kv_heads, s.page, 4), dtype=torch.float16, device="cuda"),
            s.table, s.lens)


class Step:
    """The buffers of steps of up to T tokens, up to max_n of them from one request."""

    def __init__(self, s, T, max_n):
        half = lambda *shape: torch.zeros(shape, dtype=torch.float16, device="cuda")  # noqa: E731
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        self.T, self.max_n = T, max_n
        self.new, self.release = i32(s.batch), i32(s.batch)
        self.starts, self.positions = i32(s.batch + 1), i32(T)
        self.slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.x = half(T, s.hidden)  # the residual stream: the tokens in, their hidden states out
        self.sub = half(T, s.hidden)  # what a sublayer adds to it
        self.codes = torch.zeros((T, s.hidden), dtype=torch.int8, device="cuda")
        self.scales = torch.zeros(T, device="cuda")
        self.qkv = half(T, (s.heads + 2 * s.kv_heads) * s.dim)
        self.context = half(T, s.heads, s.dim)
        self.gate_up = half(T, 2 * s.inner)
        first = s.layers[0]  # the largest of what the layers' products need
        self.products = max((bcq.new_int_workspace(T, *w.shape) for w, _ in (
            first.qkv, first.out, first.gate_up, first.down)), key=len)
        self.reserve = bcq.new_kv_reserve_workspace(s.layers[0].cache)
        self.attend = bcq.new_kv_packed_workspace(s.layers[0].cache, T, s.heads, max_n,
                                                  shared_pages=s.shared_pages)


class Server:
    """``batch`` places for requests over ``pages`` pages of every layer's cache."""

    def __init__(self, batch, pages, tokens, layers=2, hidden=4096, heads=32, kv_heads=8, dim=128,
                 inner=14336, page=64, seed=0):
        self.batch, self.pages, self.page, self.shared_pages = batch, pages, page, 0
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.inner = inner
        # one table, one stack of free pages and one set of lengths for all layers
        cache, self.free, self.count = bcq.KVCache.pool(batch, tokens, pages, 1, 64, page)
        self.table, self.lens = cache.page_table, cache.lens
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(self, g) for _ in range(layers)]

    def run(self, s):
        """One step of what s.new, s.release and s.x hold; s.x becomes the hidden states."""
        bcq.bcq_kv_reserve(self.layers[0].cache, s.new, self.free, self.count, s.starts, s.slots,
                           s.positions, release=s.release, shared_pages=self.shared_pages,
                           workspace=s.reserve)
        added = None
        for layer in self.layers:
            self.attention(layer, s, added)
            self.feed_forward(layer, s)
            added = s.sub
        s.x.add_(s.sub)
        return s.x

    def attention(self, layer, s, added):
        bcq.bcq_rms_norm(s.x, layer.norms[0], EPS, residual=added, H=s.x, codes=s.codes,
                         scales=s.scales)
        bcq.bcq_int_gemm(s.codes, s.scales, *layer.qkv, s.qkv, workspace=s.products)
        heads = (self.heads, self.kv_heads, self.kv_heads)
        q, k, v = s.qkv.view(s.T, sum(heads), self.dim).split(heads, dim=1)
        bcq.bcq_kv_append_slots(layer.cache, k, v, s.slots)
        bcq.bcq_kv_attend_packed(layer.cache, q, s.context, s.starts, s.max_n,
                                 shared_pages=self.shared_pages, workspace=s.attend)
        bcq.bcq_int_linear(s.context.flatten(1), *layer.out, s.sub, workspace=s.products)

    def feed_forward(self, layer, s):
        bcq.bcq_rms_norm(s.x, layer.norms[1], EPS, residual=s.sub, H=s.x, codes=s.codes,
                         scales=s.scales)
        bcq.bcq_int_gemm(s.codes, s.scales, *layer.gate_up, s.gate_up, workspace=s.products)
        gate, up = s.gate_up.chunk(2, dim=1)
        bcq.bcq_int_linear(torch.nn.functional.silu(gate) * up, *layer.down, s.sub,
                           workspace=s.products)

    def common(self, x):
        """Reads a prompt common to all requests, x [n][hidden] of whole pages, into pages that
        every table then begins with; before any request is served."""
        n = len(x)
        if n % self.page:
            raise ValueError("a common prompt of %d tokens, pages of %d" % (n, self.page))
        if self.lens.any():
            raise ValueError("a common prompt where tokens are cached")
        # a step leaves a request out that there is no room for
        if n > self.page * min(self.table.shape[1], int(self.count)):
            raise ValueError("a common prompt of %d tokens, %d free pages of %d and room for %d in a "
                             "table" % (n, int(self.count), self.page, self.table.shape[1]))
        s = Step(self, n, n)
        s.x.copy_(x)
        s.new[0] = n
        self.run(s)
        self.shared_pages = n // self.page
        self.table[:, :self.shared_pages] = self.table[0, :self.shared_pages].clone()
        self.lens.fill_(n)
        return s.x


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--common", type=int, default=1024)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    page = 64
    tokens = a.common + a.prompt + a.steps + 8
    server = Server(a.batch, a.common // page + a.batch * (-(-tokens // page)), tokens, a.layers)
    server.common(torch.randn((a.common, server.hidden), device="cuda").half())

    prompts = [1 + i * a.prompt // a.batch for i in range(a.batch)]  # of unlike lengths
    first = Step(server, sum(prompts), max(prompts))
    first.new.copy_(torch.tensor(prompts))
    first.x.normal_()
    hidden = server.run(first)

    one = Step(server, a.batch, 1)
    one.new.fill_(1)
    one.x.copy_(hidden[first.starts[1:].long() - 1])  # each request's last token
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        server.run(one)

    def run(steps):
        start = time.perf_counter()
        for _ in range(steps):
            graph.replay()
            one.x.copy_(one.x / one.x.float().pow(2).mean(1, keepdim=True).sqrt().half())
        torch.cuda.synchronize()
        return (time.perf_counter() - start) / steps * 1e6

    run(1)  # the first brings graph and kernels to the device
    us = run(a.steps)
    print("%d steps of %d requests through %d layers, %.1f us each; lengths %d to %d, %d of %d pages "
          "free" % (a.steps, a.batch, a.layers, us, int(server.lens.min()), int(server.lens.max()),
                    int(server.count), server.pages))
    assert torch.isfinite(one.x).all()


if __name__ == "__main__":
    main()
