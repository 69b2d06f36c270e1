"""bcq_rms_norm on the GPU against its definition: h, codes and scales to the bit, y within its
roundings."""

import sys

import numpy as np
import pytest

from oracle import lowbit as lb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import binary_coded_precision_amd as bcq  # noqa: E402

DT = {"f16": np.float16, "f32": np.float32}
EPS = 1e-5


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def padded(a, fill, extra=0):
    """A device copy of [T][K] in rows padded to 16 elements (and extra), and its whole buffer."""
    T, K = a.shape
    whole = np.full((T, (K + 15) // 16 * 16 + extra), fill, a.dtype)
    whole[:, :K] = a
    whole = torch.from_numpy(whole).cuda()
    return whole[:, :K], whole


def outputs(T, K, dtype, fill=7):
    z = np.full((T, K), fill, DT[dtype])
    return padded(z, fill), padded(z, fill, 16), padded(np.full((T, K), fill, np.int8), fill, 16), \
        torch.full((T,), 7.0, device="cuda")


def check(x, r, gamma, eps, dtype, H, Y, codes, scales):
    h, y, q, s = lb.rms_norm(x, r, gamma, eps)
    K = x.shape[1]
    if H is not None:
        np.testing.assert_array_equal(H[0].cpu().numpy(), h)
    if Y is not None:
        got = Y[0].cpu().numpy().astype(np.float64)
        # inv and two products, each rounded to fp32, then the output's type
        u = (2.0**-11 if dtype == "f16" else 0) + 3 * 2.0**-24 * 1.01
        fine = np.isfinite(y)
        tiny = 2.0**-24 if dtype == "f16" else 2.0**-148
        lim = np.finfo(DT[dtype]).max
        past = np.abs(y) >= lim * (1 + np.finfo(DT[dtype]).eps / 4)
        y[past] = np.copysign(np.inf, y[past])
        fine &= np.isfinite(y)
        assert (np.isnan(got) == np.isnan(y)).all()
        assert (got[~fine & ~np.isnan(y)] == y[~fine & ~np.isnan(y)]).all()
        assert (np.abs(got - y)[fine] <= (u * np.abs(y) + tiny)[fine]).all()
    if codes is not None:
        np.testing.assert_array_equal(scales.cpu().numpy(), s)
        np.testing.assert_array_equal(codes[0].cpu().numpy(), q)
        whole = codes[1].cpu().numpy()
        end = (K + 15) // 16 * 16
        assert (whole[:, K:end] == 0).all() and (whole[:, end:] == 7).all()
    for out in (H, Y):  # nothing behind a row
        if out is not None:
            assert (out[1][:, K:] == 7).all()


SIZES = [(1, 1), (3, 7), (2, 8), (5, 16), (67, 100), (4, 500), (3, 512), (9, 1001), (2, 2047),
         (1, 2048), (3, 2056), (1, 4096), (130, 4096), (2, 4100), (2, 8192), (3, 8193), (1, 14336),
         (2, 16385), (1, 32768), (2, 40001), (1, 131071)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T,K", SIZES)
def test_norm(T, K, dtype):
    say("rms_norm", T, K, dtype)
    rng = np.random.default_rng(T * 7 + K)
    x = rng.normal(size=(T, K)).astype(DT[dtype])
    r = (rng.normal(size=(T, K)) * np.where(rng.random(K) < 0.01, 20, 1)).astype(DT[dtype])
    gamma = (1 + 0.3 * rng.normal(size=K)).astype(DT[dtype])
    X, R = padded(x, np.nan)[0], padded(r, np.nan, 16)[0]
    G = torch.from_numpy(gamma).cuda()
    H, Y, codes, scales = outputs(T, K, dtype)
    bcq.bcq_rms_norm(X, G, EPS, residual=R, H=H[0], Y=Y[0], codes=codes[0], scales=scales)
    torch.cuda.synchronize()
    check(x, r, gamma, EPS, dtype, H, Y, codes, scales)
    # each output by itself, and without a residual
    H, Y, codes, scales = outputs(T, K, dtype)
    bcq.bcq_rms_norm(X, G, EPS, residual=R, H=H[0])
    bcq.bcq_rms_norm(X, G, EPS, Y=Y[0])
    bcq.bcq_rms_norm(X, G, EPS, codes=codes[0], scales=scales)
    torch.cuda.synchronize()
    check(x, r, gamma, EPS, dtype, H, None, None, None)
    check(x, None, gamma, EPS, dtype, None, Y, codes, scales)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T,K", [(2, 64), (3, 1001), (5, 4096), (1, 12000), (2, 40001)])
@pytest.mark.parametrize("into", ["X", "residual"])
def test_in_place(T, K, dtype, into):
    say("rms_norm in place", T, K, dtype, into)
    rng = np.random.default_rng(K)
    x = rng.normal(size=(T, K)).astype(DT[dtype])
    r = rng.normal(size=(T, K)).astype(DT[dtype])
    gamma = rng.normal(size=K).astype(DT[dtype])
    X, R = padded(x, 7), padded(r, 7)
    H = X if into == "X" else R
    _, Y, codes, scales = outputs(T, K, dtype)
    bcq.bcq_rms_norm(X[0], torch.from_numpy(gamma).cuda(), EPS, residual=R[0], H=H[0], Y=Y[0],
                     codes=codes[0], scales=scales)
    torch.cuda.synchronize()
    check(x, r, gamma, EPS, dtype, H, Y, codes, scales)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("K", [65, 4096, 40001])
def test_rows_of_any_size(K, dtype):
    """Zeros, infinities, NaN, the type's largest and smallest values, beside ordinary rows."""
    say("rms_norm sizes", K, dtype)
    rng = np.random.default_rng(K)
    big = float(np.finfo(DT[dtype]).max)
    x = rng.normal(size=(10, K)).astype(DT[dtype])
    r = np.zeros_like(x)
    x[0] = 0
    x[1, K // 2] = np.inf
    x[2, K - 1] = np.nan
    x[3] = np.where(x[3] > 0, big, -big)
    x[4] = (x[4].astype(np.float64) * float(np.finfo(DT[dtype]).tiny)).astype(DT[dtype])
    x[5], r[5] = big, big  # the sum is past the type's range
    x[6, 0] = -np.inf
    x[7] = 0
    x[7, K // 3] = big / 4
    gamma = rng.normal(size=K).astype(DT[dtype])
    H, Y, codes, scales = outputs(10, K, dtype)
    bcq.bcq_rms_norm(padded(x, np.nan)[0], torch.from_numpy(gamma).cuda(), 1e-12,
                     residual=padded(r, np.nan)[0], H=H[0], Y=Y[0], codes=codes[0], scales=scales)
    torch.cuda.synchronize()
    check(x, r, gamma, 1e-12, dtype, H, Y, codes, scales)


def test_feeds_the_integer_product():
    """Norm, then the 8-bit product: what quantizing the normed rows and multiplying gives."""
    T, K, M = 37, 1000, 260
    say("rms_norm to int_gemm", T, K, M)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, K), generator=g, device="cuda")
    gamma = torch.rand(K, generator=g, device="cuda") + 0.5
    w, ws = bcq.bcq_int_quantize(torch.randn((M, K), generator=g, device="cuda"))
    codes = torch.empty((T, 1008), dtype=torch.int8, device="cuda")[:, :K]
    scales = torch.empty(T, device="cuda")
    y = torch.empty((T, K), device="cuda")
    bcq.bcq_rms_norm(x, gamma, EPS, Y=y, codes=codes, scales=scales)
    q, s = bcq.bcq_int_quantize(y)
    assert torch.equal(q, codes) and torch.equal(s, scales)
    a, b = torch.empty((2, T, M), device="cuda")
    bcq.bcq_int_gemm(codes, scales, w, ws, a)
    bcq.bcq_int_linear(y, w, ws, b)
    assert torch.equal(a, b)


def test_no_rows():
    e = torch.empty((0, 64), device="cuda")
    bcq.bcq_rms_norm(e, torch.ones(64, device="cuda"), EPS, H=e)


def test_more_long_rows_than_a_launch_has_room_for():
    """Long rows take 1024 work items each, of which a launch has less than 2^32."""
    T, K = (1 << 22) + 1, 8200
    say("rms_norm", T, K)
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("takes 104 GB of device memory")
    x = torch.empty((T, 8208), dtype=torch.float16, device="cuda")
    codes = torch.full((T, 8208), 7, dtype=torch.int8, device="cuda")
    scales = torch.full((T,), 7.0, device="cuda")
    gamma = torch.ones(K, dtype=torch.float16, device="cuda")
    x[:] = torch.randn(8208, dtype=torch.float16, device="cuda")
    bcq.bcq_rms_norm(x[:, :K], gamma, EPS, codes=codes[:, :K], scales=scales)
    check(x[:1, :K].cpu().numpy(), None, gamma.cpu().numpy(), EPS, "f16", None, None,
          (codes[:1, :K], codes[:1]), scales[:1])
    assert (scales == scales[0]).all()
    for rows in codes.split(1 << 16):
        assert (rows == codes[0]).all()
    del x, codes
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,K", [(4095, 1000), (4097, 1000), (4099, 513), (4101, 72), (4096, 1024),
                                 (256, 4096), (257, 4096), (300, 2050), (257, 8191)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_many_rows(T, K, dtype):
    test_norm(T, K, dtype)
