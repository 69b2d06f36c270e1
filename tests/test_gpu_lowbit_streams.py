"""The low-bit operators' own allocations on the GPU, with work pending on other streams."""

import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def busy(product):
    """A few milliseconds of work on the current stream."""
    for _ in range(20):
        product @ product


def test_calls_on_two_streams_with_workspaces_of_their_own():
    """Products on the current stream and on another, the second queued while the first waits:
    each finds its codes and sums as it left them."""
    say("int_linear on two streams")
    T, M, K = 100, 100, 4096  # codes, scales and the sums of K's slices in the workspace
    x = torch.randn((2, T, K), device="cuda", dtype=torch.float16)
    w = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8)
    s = torch.full((M,), 0.01, device="cuda")
    want, got = (torch.empty((2, T, M), device="cuda", dtype=torch.float16) for _ in range(2))
    for i in (0, 1):
        bcq.bcq_int_linear(x[i], w, s, want[i])
    big = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        got.zero_()
        torch.cuda.synchronize()
        busy(big)
        bcq.bcq_int_linear(x[0], w, s, got[0])
        bcq.bcq_int_linear(x[1], w, s, got[1], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_attention_on_two_streams_with_workspaces_of_their_own():
    say("kv_attend on two streams")
    c = bcq.KVCache.new(1, 4096, 2, 64)
    c.lens.fill_(4000)
    v = torch.randn((2, 1, 4000, 2, 64), device="cuda")
    bcq.bcq_kv_append(c, v[0], v[1])
    q = torch.randn((2, 1, 1, 4, 64), device="cuda")
    want, got = torch.empty_like(q), torch.empty_like(q)
    for i in (0, 1):
        bcq.bcq_kv_attend(c, q[i], want[i])
    big = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        got.zero_()
        torch.cuda.synchronize()
        busy(big)
        bcq.bcq_kv_attend(c, q[0], got[0])
        bcq.bcq_kv_attend(c, q[1], got[1], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_the_quantizers_outputs_dropped_before_it_has_run():
    """What the current stream allocates next is not what another stream is still to write."""
    say("int_quantize on another stream")
    x = torch.randn((512, 4096), device="cuda", dtype=torch.float16)
    big = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy(big)
    codes, scales = bcq.bcq_int_quantize(x, stream=side)
    shape, n = codes.shape, len(scales)
    del codes, scales
    mine = torch.full(shape, 3, dtype=torch.int8, device="cuda")
    ones = torch.ones(n, device="cuda")
    torch.cuda.synchronize()
    assert (mine == 3).all() and (ones == 1).all()
