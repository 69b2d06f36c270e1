"""The Python binding of the norm and of the packed step's operators by itself (no GPU), as
test_lowbit_binding looks at the others: what is allocated, where, and with which device current."""

import pytest

torch = pytest.importorskip("torch")

from binary_coded_precision_amd import lowbit  # noqa: E402
from test_lowbit_binding import OnDevice, Stream, cache, machine, zeros  # noqa: E402, F401

f32, i32, i64, i8, u8 = torch.float32, torch.int32, torch.int64, torch.int8, torch.uint8

# each call: its entry point, plain arguments, tensors as (shape, dtype)
NORM = (lowbit.bcq_rms_norm, dict(eps=1e-5),
        dict(X=((3, 64), f32), gamma=((64,), f32), residual=((3, 64), f32), H=((3, 64), f32),
             Y=((3, 64), f32), codes=((3, 64), i8), scales=((3,), f32)))
RESERVE = (lowbit.bcq_kv_reserve, dict(cache=None),
           dict(new_tokens=((1,), i32), free_pages=((2,), i32), free_count=((1,), i32),
                starts=((2,), i32), slots=((5,), i64), positions=((5,), i32),
                release=((1,), i32), lens_out=((1,), i32), page_table_out=((1, 2), i32),
                free_pages_out=((2,), i32), free_count_out=((1,), i32), workspace=((4096,), u8)))
VECTORS = dict(K=((5, 1, 64), f32), V=((5, 1, 64), f32), slots=((5,), i64))
APPEND = (lowbit.bcq_kv_append_slots, dict(cache=None), VECTORS)
READ = (lowbit.bcq_kv_read_slots, dict(cache=None), VECTORS)
ATTEND = (lowbit.bcq_kv_attend_packed, dict(cache=None, max_n=5),
          dict(Q=((5, 2, 64), f32), O=((5, 2, 64), f32), starts=((2,), i32),
               workspace=((4096,), u8)))
CALLS = [NORM, RESERVE, APPEND, READ, ATTEND]


def call(what, index=0, away=None, stream=None, leave=(), **change):
    fn, plain, tensors = what
    args = {n: cache(index) if n == "cache" else v for n, v in plain.items()}
    for n, (shape, dtype) in tensors.items():
        if n not in leave:
            args[n] = zeros(*shape, dtype=dtype, index=1 - index if n == away else index)
    args.update(change)
    fn(**args, stream=stream)


def name(what):
    return what[0].__name__


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("what", CALLS, ids=name)
def test_a_call_runs_with_its_tensors_device_current(machine, what, index):  # noqa: F811
    call(what, index)
    (called, args, device), = machine.calls
    assert (called, args[-1], device) == (name(what), 100 + index, index)
    assert machine.device == 0 and not machine.allocated


@pytest.mark.parametrize("what", CALLS, ids=name)
def test_a_stream_of_another_device_is_refused(machine, what):  # noqa: F811
    with pytest.raises(ValueError, match="stream"):
        call(what, stream=Stream(7, 1))
    assert not machine.calls


@pytest.mark.parametrize("what", CALLS, ids=name)
def test_tensors_of_two_devices_are_refused(machine, what):  # noqa: F811
    for away in what[2]:
        with pytest.raises(ValueError, match="device"):
            call(what, away=away)
        assert not machine.calls, away


@pytest.mark.parametrize("what", [RESERVE, ATTEND], ids=name)
def test_a_workspace_is_memory_of_the_stream_it_is_used_on(machine, what):  # noqa: F811
    side = Stream(7)
    call(what, stream=side, leave=("workspace",))
    assert machine.allocated == [(side, 0)]
    assert machine.calls[0][0] == name(what) and machine.calls[0][1][-1] == 7


@pytest.mark.parametrize("what", [RESERVE, ATTEND], ids=name)
@pytest.mark.parametrize("bad", ["host", "strided"])
def test_a_workspace_that_kernels_cannot_write_is_refused(machine, what, bad):  # noqa: F811
    w = torch.zeros(1 << 13, dtype=u8)
    if bad == "strided":
        w = OnDevice(w[:16].expand(512, 16))
    with pytest.raises(ValueError, match="workspace"):
        call(what, workspace=w)
    assert not machine.calls


@pytest.mark.parametrize("what,change", [
    (NORM, dict(Y=(3, 65))), (NORM, dict(residual=(2, 64))), (NORM, dict(gamma=(63,))),
    (NORM, dict(scales=(4,))), (NORM, dict(codes=(3, 63))), (NORM, dict(X=(3, 64, 1))),
    (RESERVE, dict(new_tokens=(2,))), (RESERVE, dict(free_pages=(3,))),
    (RESERVE, dict(starts=(1,))), (RESERVE, dict(positions=(4,))), (RESERVE, dict(slots=(5, 1))),
    (RESERVE, dict(page_table_out=(2, 1))), (RESERVE, dict(release=(1, 1))),
    (APPEND, dict(K=(5, 2, 64))), (APPEND, dict(V=(4, 1, 64))), (APPEND, dict(slots=(4,))),
    (READ, dict(K=(5, 1, 32))), (ATTEND, dict(Q=(5, 2, 32))), (ATTEND, dict(O=(4, 2, 64))),
    (ATTEND, dict(starts=(3,))), (ATTEND, dict(Q=(1, 5, 2, 64))),
], ids=lambda v: name(v) if isinstance(v, tuple) else "-".join(v))
def test_other_shapes_are_refused(machine, what, change):  # noqa: F811
    (n, shape), = change.items()
    with pytest.raises(ValueError):
        call(what, **{n: zeros(*shape, dtype=what[2][n][1])})
    assert not machine.calls


@pytest.mark.parametrize("what,n,dtype", [
    (NORM, "Y", torch.float16), (NORM, "gamma", torch.float16), (NORM, "codes", u8),
    (NORM, "X", torch.float64), (RESERVE, "new_tokens", i64), (RESERVE, "slots", i32),
    (APPEND, "V", torch.float16), (APPEND, "slots", i32), (ATTEND, "O", torch.float16),
    (ATTEND, "starts", i64), (ATTEND, "Q", torch.bfloat16),
], ids=lambda v: name(v) if isinstance(v, tuple) else str(v))
def test_other_types_are_refused(machine, what, n, dtype):  # noqa: F811
    with pytest.raises((ValueError, TypeError)):
        call(what, **{n: zeros(*what[2][n][0], dtype=dtype)})
    assert not machine.calls


def test_strided_channels_are_refused(machine):  # noqa: F811
    wide = OnDevice(torch.zeros(5, 2, 128)[:, :, ::2])
    one = OnDevice(torch.zeros(5, 1, 128)[:, :, ::2])
    for c, n, t in ((ATTEND, "Q", wide), (ATTEND, "O", wide), (APPEND, "K", one), (READ, "V", one),
                    (NORM, "H", OnDevice(torch.zeros(3, 128)[:, ::2]))):
        with pytest.raises(ValueError):
            call(c, **{n: t})
    assert not machine.calls
