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


# ----------------------------------------------------------------------------- devices


def entries(index):
    """Every call of the binding on tensors of one device, as functions of a stream."""
    k, c = zeros(1, 1, 1, 64, index=index), cache(index)
    return {
        "bcq_int_quantize": lambda t: lowbit.bcq_int_quantize(zeros(3, 64, index=index), stream=t),
        "bcq_kv_append": lambda t: lowbit.bcq_kv_append(c, k, k, stream=t),
        "bcq_kv_read": lambda t: lowbit.bcq_kv_read(c, k, k, stream=t),
        **with_workspace(index),
    }


ENTRIES = WITH_WORKSPACE + ("bcq_int_quantize", "bcq_kv_append", "bcq_kv_read")


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_runs_with_its_tensors_device_current(machine, name, index):
    """A launch goes to the current device, whose streams alone it may name."""
    entries(index)[name](None)
    (called, args, device), = machine.calls
    assert (called, args[-1], device) == (name, 100 + index, index)
    assert machine.device == 0 and all(d == index for _, d in machine.allocated)


@pytest.mark.parametrize("name", ENTRIES)
def test_a_stream_of_another_device_is_refused(machine, name):
    with pytest.raises(ValueError, match="stream"):
        entries(0)[name](Stream(7, 1))
    assert not machine.calls and not machine.allocated


def test_tensors_of_two_devices_are_refused(machine):
    f32, i32, i8, u8 = torch.float32, torch.int32, torch.int8, torch.uint8
    here, c = 0, cache(0)
    # each call with its tensors, one of which at a time is on the other device
    calls = [
        (lowbit.bcq_int_quantize, dict(X=(3, 64)), {},
         dict(codes=((3, 64), i8), scales=((3,), f32))),
        (lowbit.bcq_int_gemm, {}, {},
         dict(A=((3, 64), i8), a_scales=((3,), f32), W=((4, 64), i8), w_scales=((4,), f32),
              Y=((3, 4), f32), bias=((4,), f32), workspace=((4096,), u8))),
        (lowbit.bcq_int_linear, {}, {},
         dict(X=((3, 64), f32), W=((4, 64), i8), w_scales=((4,), f32), Y=((3, 4), f32),
              bias=((4,), f32), workspace=((4096,), u8))),
        (lowbit.bcq_kv_append, {}, dict(cache=c),
         dict(K=((1, 1, 1, 64), f32), V=((1, 1, 1, 64), f32), positions=((1, 1), i32),
              weights=((1, 1, 32), f32), pos=((1, 1, 32), i32))),
        (lowbit.bcq_kv_read, {}, dict(cache=c),
         dict(K=((1, 1, 1, 64), f32), V=((1, 1, 1, 64), f32))),
        (lowbit.bcq_kv_attend, {}, dict(cache=c),
         dict(Q=((1, 1, 1, 64), f32), O=((1, 1, 1, 64), f32), weights=((1, 1, 32), f32),
              workspace=((4096,), u8))),
        (lowbit.bcq_kv_evict, {}, dict(cache=c, keep=5, recent=1),
         dict(weights=((1, 1, 32), f32), pos=((1, 1, 32), i32), lens_out=((1,), i32),
              weights_out=((1, 1, 32), f32), pos_out=((1, 1, 32), i32),
              workspace=((4096,), u8))),
    ]
    for fn, plain, more, tensors in calls:
        def arguments(away):
            got = {n: zeros(*shape) for n, shape in plain.items()}
            for n, (shape, dtype) in tensors.items():
                got[n] = zeros(*shape, dtype=dtype, index=1 if n == away else here)
            return dict(got, **more)

        fn(**arguments(None))
        machine.calls.clear()
        for away in tensors:
            with pytest.raises(ValueError, match="device"):
                fn(**arguments(away))
            assert not machine.calls, (fn.__name__, away)


def test_a_cache_lies_on_one_device(machine):
    shapes = [((2, 1, 16, 32), torch.uint8), ((2, 1, 4, 128), torch.uint8),
              ((2, 1, 16, 4), torch.float16), ((1, 2), torch.int32), ((1,), torch.int32)]
    for away in range(5):
        with pytest.raises(ValueError, match="device"):
            lowbit.KVCache(*(zeros(*shape, dtype=dtype, index=int(i == away))
                             for i, (shape, dtype) in enumerate(shapes)))
