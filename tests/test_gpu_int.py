"""The 8-bit integer linear layer on the GPU against its float64 definition.  Codes and scales
are defined to the bit; outputs differ from exact integer sums only by single-precision
scaling and the one rounding to the output type."""

import sys

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402

DT = {"f16": (torch.float16, np.float16), "f32": (torch.float32, np.float32)}


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def rows(x, dtype):
    """A device matrix whose rows start at multiples of 16 bytes, NaN between them."""
    t, k = x.shape
    pad = torch.full((t, (k + 15) // 16 * 16 + 16), float("nan"), dtype=DT[dtype][0],
                     device="cuda")
    pad[:, :k] = torch.from_numpy(x).cuda()
    return pad[:, :k]


def weights(w, fill=77):
    """Codes with rows of whole 16 bytes, other codes between them."""
    m, k = w.shape
    pad = torch.full((m, (k + 15) // 16 * 16), fill, dtype=torch.int8, device="cuda")
    pad[:, :k] = torch.from_numpy(w).cuda()
    return pad[:, :k]


def tolerance(y, bias, dtype):
    # scale product, times the sum (converted once), plus the bias: 4 roundings of 2^-24, and
    # one to the output's type
    mag = np.abs(y) + (0 if bias is None else 2 * np.abs(bias.astype(np.float64)))
    return 4 * 2.0**-24 * mag + (2.0**-11 * np.abs(y) + 2.0**-25 if dtype == "f16" else 0)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 7), (5, 16), (2, 129), (33, 1001), (4, 4096),
                                 (7, 14336), (1, 20000)])
def test_quantize_is_exact(T, K, dtype):
    say("int_quantize", T, K, dtype)
    rng = np.random.default_rng(T * K)
    x = (rng.normal(size=(T, K)) * 10.0 ** rng.integers(-3, 3, (T, 1))).astype(DT[dtype][1])
    if T > 2:
        x[1] = 0
        x[2, K // 2] = 3e4
    codes, scales = bcq.bcq_int_quantize(rows(x, dtype))
    c, s = lb.quantize_rows(x)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    whole = torch.as_strided(codes, (T, (K + 15) // 16 * 16), (codes.stride(0), 1))
    assert not whole[:, K:].any()  # what pads a row is zero


def test_quantize_of_what_is_not_finite():
    x = np.ones((3, 40), np.float32)
    x[0, 3], x[1, 39] = np.inf, np.nan
    codes, scales = bcq.bcq_int_quantize(rows(x, "f32"))
    assert torch.isnan(scales[:2]).all() and not codes[:2].any() and scales[2] == np.float32(1 / 127)


SHAPES = [(1, 1, 1), (1, 5, 64), (1, 16, 128), (1, 100, 1000), (1, 4096, 4096), (2, 40, 4096),
          (4, 33, 4096), (3, 17, 5000), (1, 7, 16384), (1, 7, 16385), (16, 31, 1024),
          (17, 64, 512), (16, 48, 1040), (37, 300, 700), (64, 64, 128), (65, 129, 257),
          (128, 128, 1001), (200, 1000, 96), (9, 1025, 14336), (515, 260, 333),
          (1030, 2050, 130)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T,M,K", SHAPES)
def test_linear(T, M, K, dtype):
    say("int_linear", T, M, K, dtype)
    rng = np.random.default_rng(T + M + K)
    x = rng.normal(size=(T, K)).astype(DT[dtype][1])
    w = rng.integers(-128, 128, (M, K)).astype(np.int8)
    ws = (rng.random(M).astype(np.float32) + 0.5) / 1024
    bias = rng.normal(size=M).astype(DT[dtype][1]) if (T + M) % 2 else None
    y = torch.full((T + 1, M + 3), 7.0, dtype=DT[dtype][0], device="cuda")
    wd, sd = weights(w), torch.from_numpy(ws).cuda()
    bd = None if bias is None else torch.from_numpy(bias).cuda()
    bcq.bcq_int_linear(rows(x, dtype), wd, sd, y[:T, :M], bias=bd)
    c, s = lb.quantize_rows(x)
    ref = lb.product(c, s, w, ws, bias)
    got = y.cpu().numpy().astype(np.float64)
    assert (np.abs(got[:T, :M] - ref) <= tolerance(ref, bias, dtype)).all()
    assert (got[T:] == 7).all() and (got[:, M:] == 7).all()
    # the two steps by themselves give the same bits
    z = torch.empty((T, M), dtype=DT[dtype][0], device="cuda")
    codes, scales = bcq.bcq_int_quantize(rows(x, dtype))
    bcq.bcq_int_gemm(codes, scales, wd, sd, z, bias=bd)
    assert torch.equal(z, y[:T, :M])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T,M,K", [
    (3, 50, 5461), (20, 70, 4100), (40, 64, 5000), (64, 8000, 1040),  # few tokens, K split or not
    (100, 100, 4096), (300, 257, 2049),  # the small tile, K split
    (1001, 4000, 160), (4090, 4104, 144),  # the larger tiles, outputs of whole 16 bytes
    (4100, 5104, 144)])  # the last of 340 tiles in halves, some of them past the tokens
def test_linear_by_way(T, M, K, dtype):
    test_linear(T, M, K, dtype)


def test_extreme_codes_do_not_overflow():
    K = 131071
    a = torch.full((2, K + 1), -128, dtype=torch.int8, device="cuda")
    a[:, K:] = 0
    y = torch.empty((2, 2), dtype=torch.float32, device="cuda")
    one = torch.ones(2, device="cuda")
    bcq.bcq_int_gemm(a[:, :K], one, a[:, :K], one, y)
    assert (y == float(np.float32(128 * 128 * K))).all()


@pytest.mark.parametrize("T,K", [(2, 64), (40, 700)])
def test_rows_that_are_not_finite_stay_alone(T, K):
    x = np.ones((T, K), np.float32)
    x[1, K - 1] = np.inf
    y = torch.zeros((T, 20), device="cuda")
    bcq.bcq_int_linear(rows(x, "f32"), weights(np.ones((20, K), np.int8)),
                       torch.ones(20, device="cuda"), y)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def test_no_tokens():
    w = weights(np.ones((4, 32), np.int8))
    y = torch.empty((0, 4), device="cuda")
    bcq.bcq_int_linear(torch.empty((0, 32), device="cuda"), w, torch.ones(4, device="cuda"), y)


@pytest.mark.parametrize("T", [1, 40])
def test_captured_and_on_another_stream(T):
    rng = np.random.default_rng(T)
    M, K = 96, 640
    w = rng.integers(-127, 128, (M, K)).astype(np.int8)
    wd, sd = weights(w), torch.full((M,), 0.01, device="cuda")
    x = torch.empty((T, K), dtype=torch.float16, device="cuda")
    y = torch.empty((T, M), dtype=torch.float16, device="cuda")
    ws = bcq.new_int_workspace(T, M, K)
    x.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bcq.bcq_int_linear(x, wd, sd, y, stream=side)  # the workspace is the allocator's
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bcq.bcq_int_linear(x, wd, sd, y, workspace=ws)
    for i in range(4):
        x.normal_()
        want = torch.empty_like(y)
        bcq.bcq_int_linear(x, wd, sd, want)
        y.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
