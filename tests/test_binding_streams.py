"""What the products' binding allocates for a call on a given stream (no GPU), through the
stand-ins of test_lowbit_binding."""

import pytest

import binary_coded_precision_amd as bcq
from test_lowbit_binding import Stream, machine, zeros  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.fixture
def calls(machine, monkeypatch):  # noqa: F811
    """The calls that allocate device memory, as functions of a stream."""
    monkeypatch.setattr(bcq, "_lib", machine)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(100))
    M, K, i32 = 16, 128, torch.int32
    table = zeros(2, M, 1), zeros(M, 1)
    store = bcq.Store(M, K, 2, zeros(1 << 10, dtype=i32), {2: table[0]}, {2: table[1]})
    x, y = zeros(1, K), zeros(1, M)
    u, v, alpha = zeros(M, 1, dtype=i32), zeros(8, K // 32, dtype=i32), zeros(8)
    signs = zeros(2, M, K // 32, dtype=i32)
    return {
        "bcq_gemm_skinny": (1, lambda s: bcq.bcq_gemm_skinny(store, 2, x, y, stream=s)),
        "bcq_gemv_mixed_p": (1, lambda s: bcq.bcq_gemv_mixed_p(store, [2], x, y, stream=s)),
        "bcq_lowrank_correct": (1, lambda s: bcq.bcq_lowrank_correct(u, v, alpha, x[0], y[0],
                                                                     stream=s)),
        "bcq_gemv_lowrank": (1, lambda s: bcq.bcq_gemv_lowrank(store, 2, x[0], u, v, alpha, y[0],
                                                               stream=s)),
        "bcq_quantize": (3, lambda s: bcq.bcq_quantize(zeros(M, K), 2, stream=s)),
        "bcq_pack_planes": (1, lambda s: bcq.Store.from_quantized(signs, {2: table[0]},
                                                                  {2: table[1]}, stream=s)),
    }


@pytest.mark.parametrize("name", ["bcq_gemm_skinny", "bcq_gemv_mixed_p", "bcq_lowrank_correct",
                                  "bcq_gemv_lowrank", "bcq_quantize", "bcq_pack_planes"])
def test_allocations_are_memory_of_the_stream_they_are_used_on(machine, calls, name):  # noqa: F811
    """Memory of the current stream's may still be in use there by what was queued before it was
    freed."""
    number, call = calls[name]
    side = Stream(7)
    for stream, raw in ((side, 7), (None, 100)):
        machine.calls.clear()
        machine.allocated.clear()
        call(stream)
        assert machine.allocated == [(stream, 0)] * number
        assert machine.calls[0][0] == name and machine.calls[0][1][-1].value == raw
