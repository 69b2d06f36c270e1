"""The Python binding of the low-bit operators by itself (no GPU): what it allocates, where, and
with which device current, seen through stand-ins for device tensors and for the library."""

import contextlib

import pytest

from binary_coded_precision_amd import lowbit

torch = pytest.importorskip("torch")


class OnDevice:
    """A host tensor that says it is on a device."""

    def __init__(self, t, index=0):
        self.t, self.index = t, index
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, at):
        return OnDevice(self.t[at], self.index)

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        pass


class Stream:
    def __init__(self, raw, index=0):
        self.cuda_stream, self.device_index = raw, index


class Machine:
    """What the binding asks of torch and of the library, and what it was told."""

    def __init__(self):
        self.stream, self.device = None, 0
        self.allocated = []  # (stream current at the time, device)
        self.calls = []  # (entry point, arguments, device current at the time)

    def __getattr__(self, name):  # as the library
        def entry(*args):
            if name.endswith("_bytes"):
                return 1 << 12
            self.calls.append((name, args, self.device))
            return 0

        return entry

    @contextlib.contextmanager
    def on_stream(self, stream):
        before, self.stream = self.stream, stream
        yield
        self.stream = before

    @contextlib.contextmanager
    def on_device(self, index):
        before, self.device = self.device, index
        yield
        self.device = before


@pytest.fixture
def machine(monkeypatch):
    m = Machine()
    real = torch.empty

    def empty(*size, device=None, **kw):
        index = torch.device(device).index or 0
        m.allocated.append((m.stream, index))
        return OnDevice(real(*size, **kw), index)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", m.on_stream)
    monkeypatch.setattr(torch.cuda, "device", m.on_device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: m.device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index,
                        raising=False)
    monkeypatch.setattr(lowbit, "torch", torch)
    monkeypatch.setattr(lowbit, "_lib", m)
    return m


def zeros(*shape, dtype=torch.float16, index=0):
    return OnDevice(torch.zeros(shape, dtype=dtype), index)


def cache(index=0):
    return lowbit.KVCache(zeros(2, 1, 16, 32, dtype=torch.uint8, index=index),
                          zeros(2, 1, 4, 128, dtype=torch.uint8, index=index),
                          zeros(2, 1, 16, 4, index=index),
                          zeros(1, 2, dtype=torch.int32, index=index),
                          zeros(1, dtype=torch.int32, index=index))


def with_workspace(index=0):
    """The calls that allocate a workspace, as functions of a stream."""
    x, y = zeros(3, 64, index=index), zeros(3, 4, index=index)
    a, w = zeros(3, 64, dtype=torch.int8, index=index), zeros(4, 64, dtype=torch.int8, index=index)
    s = {n: zeros(n, dtype=torch.float32, index=index) for n in (3, 4)}
    q, c = zeros(1, 1, 1, 64, index=index), cache(index)
    weights = zeros(1, 1, 32, dtype=torch.float32, index=index)
    pos = zeros(1, 1, 32, dtype=torch.int32, index=index)
    return {
        "bcq_int_linear": lambda t: lowbit.bcq_int_linear(x, w, s[4], y, stream=t),
        "bcq_int_gemm": lambda t: lowbit.bcq_int_gemm(a, s[3], w, s[4], y, stream=t),
        "bcq_kv_attend": lambda t: lowbit.bcq_kv_attend(c, q, q, stream=t),
        "bcq_kv_evict": lambda t: lowbit.bcq_kv_evict(c, 5, 1, weights, pos, stream=t),
    }


WITH_WORKSPACE = ("bcq_int_gemm", "bcq_int_linear", "bcq_kv_attend", "bcq_kv_evict")


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_a_workspace_is_memory_of_the_stream_it_is_used_on(machine, name):
    """Memory that another stream's allocator hands out may still be in use there."""
    side = Stream(7)
    with_workspace()[name](side)
    assert machine.allocated == [(side, 0)]
    assert machine.calls[0][0] == name and machine.calls[0][1][-1] == 7


def test_the_quantizers_outputs_are_memory_of_its_stream(machine):
    """Dropped early, they may be handed out again only to what is queued behind the call."""
    side = Stream(7)
    codes, scales = lowbit.bcq_int_quantize(zeros(3, 64), stream=side)
    assert machine.allocated == [(side, 0), (side, 0)]
    assert codes.shape == (3, 64) and scales.shape == (3,)
    machine.allocated.clear()
    lowbit.bcq_int_quantize(zeros(3, 64))
    assert machine.allocated == [(None, 0), (None, 0)]


@pytest.mark.parametrize("bad", ["host", "strided"])
def test_a_workspace_that_kernels_cannot_write_is_refused(machine, bad):
    w = torch.zeros(1 << 13, dtype=torch.uint8)
    if bad == "strided":  # its bytes are fewer than its extent says
        w = OnDevice(w[:16].expand(512, 16))
    x, y = zeros(3, 64), zeros(3, 4)
    a, b = zeros(3, 64, dtype=torch.int8), zeros(4, 64, dtype=torch.int8)
    s = {n: zeros(n, dtype=torch.float32) for n in (3, 4)}
    q, c = zeros(1, 1, 1, 64), cache()
    weights, pos = zeros(1, 1, 32, dtype=torch.float32), zeros(1, 1, 32, dtype=torch.int32)
    for call in (lambda: lowbit.bcq_int_linear(x, b, s[4], y, workspace=w),
                 lambda: lowbit.bcq_int_gemm(a, s[3], b, s[4], y, workspace=w),
                 lambda: lowbit.bcq_kv_attend(c, q, q, workspace=w),
                 lambda: lowbit.bcq_kv_evict(c, 5, 1, weights, pos, workspace=w)):
        with pytest.raises(ValueError, match="workspace"):
            call()
    assert not machine.calls
