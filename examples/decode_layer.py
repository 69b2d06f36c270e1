"""The attention block of a decoder layer served in few bits, from a prompt to a bounded cache.

A prompt's projections run as 8-bit integer products (bcq_int_linear), a decode step's on the
binary-coded planes of the same weights at a precision chosen for the step (bcq_gemm_skinny).
Keys and values go into a paged 4-bit cache (bcq_kv_append), attention reads its codes and sums
the weights that each cached token receives (bcq_kv_attend), and the tokens of little weight leave
when a sequence passes its budget (bcq_kv_evict), so that a long generation runs in constant memory.
A decode step is captured once in a graph: the lengths are on the device.

    python examples/decode_layer.py [--batch 8] [--prompt 1000] [--steps 200] [--keep 512]
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import binary_coded_precision_amd as bcq  # noqa: E402


class AttentionBlock:
    """Queries, keys and values from one projection, attention over the cache, an output
    projection; random weights.  ``planes`` of the BCQ stores are used at precisions 2 and up."""

    def __init__(self, batch, hidden=4096, heads=32, kv_heads=8, head_dim=128, keep=512, recent=64,
                 longest_prompt=1024, planes=3, page_tokens=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = (heads + 2 * kv_heads) * head_dim
        weights = [torch.randn(shape, generator=g, device="cuda").mul_(hidden ** -0.5).half()
                   for shape in ((rows, hidden), (hidden, heads * head_dim))]
        self.planes = [bcq.Store.from_quantized(*bcq.bcq_quantize(w, planes)) for w in weights]
        self.codes = [bcq.bcq_int_quantize(w) for w in weights]
        self.batch, self.heads, self.kv_heads, self.head_dim = batch, heads, kv_heads, head_dim
        self.hidden, self.keep, self.recent = hidden, keep, recent
        # a step's token lies past the kept ones until the eviction that ends the step
        self.cache = bcq.KVCache.new(batch, max(keep + 1, longest_prompt), kv_heads, head_dim,
                                     page_tokens)
        self.weights, self.pos = self.cache.tracking()
        self.next = torch.zeros((batch, 1), dtype=torch.int32, device="cuda")  # positions
        self.attend_space = bcq.new_kv_workspace(self.cache, 1, heads, weights=True)
        self.evict_space = bcq.new_kv_evict_workspace(self.cache, keep)
        self.plane_spaces = [bcq.new_workspace(s, batch) for s in self.planes]

    def split(self, qkv):
        """Views [batch][n][heads][head_dim] of the projection's q, k and v."""
        t = qkv.view(self.batch, -1, self.heads + 2 * self.kv_heads, self.head_dim)
        return t.split((self.heads, self.kv_heads, self.kv_heads), dim=2)

    def prompt(self, x):
        """x [batch][n][hidden] of an empty cache -> the block's output of the same shape."""
        n = x.shape[1]
        if n > self.cache.room:
            raise ValueError("a prompt of %d tokens, room for %d" % (n, self.cache.room))
        x = x.reshape(-1, self.hidden)
        qkv = x.new_empty((len(x), self.codes[0][0].shape[0]))
        bcq.bcq_int_linear(x, *self.codes[0], qkv)
        q, k, v = self.split(qkv)
        self.cache.lens.fill_(n)
        self.next.fill_(n)
        bcq.bcq_kv_append(self.cache, k, v, weights=self.weights, pos=self.pos)
        context = q.new_empty((self.batch, n, self.heads, self.head_dim))
        bcq.bcq_kv_attend(self.cache, q, context, weights=self.weights)
        out = torch.empty_like(x)
        bcq.bcq_int_linear(context.view(len(x), -1), *self.codes[1], out)
        bcq.bcq_kv_evict(self.cache, self.keep, self.recent, self.weights, self.pos,
                         workspace=self.evict_space)
        return out.view(self.batch, n, self.hidden)

    def step(self, x, out, precision):
        """One token of every sequence: x and out [batch][hidden]."""
        qkv = x.new_empty((self.batch, self.planes[0].M))
        bcq.bcq_gemm_skinny(self.planes[0], precision, x, qkv, workspace=self.plane_spaces[0])
        q, k, v = self.split(qkv)
        self.cache.lens.add_(1)
        bcq.bcq_kv_append(self.cache, k, v, positions=self.next, weights=self.weights,
                          pos=self.pos)
        self.next.add_(1)
        context = x.new_empty((self.batch, 1, self.heads, self.head_dim))
        bcq.bcq_kv_attend(self.cache, q, context, weights=self.weights,
                          workspace=self.attend_space)
        bcq.bcq_gemm_skinny(self.planes[1], precision, context.view(self.batch, -1), out,
                            workspace=self.plane_spaces[1])
        bcq.bcq_kv_evict(self.cache, self.keep, self.recent, self.weights, self.pos,
                         workspace=self.evict_space)
        return q, context


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--keep", type=int, default=512)
    ap.add_argument("--precision", type=int, default=2, choices=(2, 3))
    a = ap.parse_args()
    block = AttentionBlock(a.batch, keep=a.keep, recent=min(64, a.keep), longest_prompt=a.prompt)
    x = torch.randn((a.batch, a.prompt, block.hidden), device="cuda").half()
    y = block.prompt(x)
    token, out = y[:, -1].contiguous(), torch.empty_like(y[:, -1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(token, out, a.precision)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
        token.copy_(out)
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / a.steps * 1e6
    pos = block.pos[0, 0, :block.cache.lens[0]]
    print("%d steps of %d sequences, %.1f us each; %d of %d tokens cached, positions %d to %d" %
          (a.steps, a.batch, us, len(pos), int(block.next[0]), int(pos.min()), int(pos.max())))
    assert torch.isfinite(out).all()


if __name__ == "__main__":
    main()
