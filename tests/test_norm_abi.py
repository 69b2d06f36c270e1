"""Refusals of bcq_rms_norm, without a GPU: every call here is rejected (or has nothing to do)
before any HIP call, so the addresses are never followed."""

import pytest

import binary_coded_precision_amd as bcq

OK, INVALID, ALIGNMENT = 0, -1, -3
F16, F32 = 1, 2
A = 4096  # an aligned address

NORM = dict(X=A, ldx=104, residual=A, ldr=104, gamma=A, eps=1e-5, T=3, K=100, dtype=F16, H=A,
            ldh=104, Y=A, ldy=104, codes=A, ldc=112, scales=A, stream=None)


@pytest.fixture(scope="module")
def lib():
    return bcq.load()


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(T=1 << 24), INVALID), (dict(K=0), INVALID),
    (dict(K=131072, ldx=131072), INVALID), (dict(dtype=0), INVALID), (dict(dtype=3), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=1e-40), INVALID),
    (dict(X=None), INVALID), (dict(gamma=None), INVALID),
    (dict(H=None, Y=None, codes=None, scales=None), INVALID),
    (dict(scales=None), INVALID), (dict(codes=None), INVALID),
    (dict(ldx=96), INVALID), (dict(ldr=96), INVALID), (dict(ldh=96), INVALID),
    (dict(ldy=96), INVALID), (dict(ldc=96), INVALID),
    (dict(X=A + 2), ALIGNMENT), (dict(residual=A + 8), ALIGNMENT), (dict(gamma=A + 4), ALIGNMENT),
    (dict(H=A + 8), ALIGNMENT), (dict(Y=A + 8), ALIGNMENT), (dict(codes=A + 8), ALIGNMENT),
    (dict(scales=A + 2), ALIGNMENT), (dict(ldx=101), ALIGNMENT), (dict(ldr=101), ALIGNMENT),
    (dict(ldh=101), ALIGNMENT), (dict(ldy=101), ALIGNMENT), (dict(ldc=120), ALIGNMENT),
    (dict(dtype=F32, ldx=102), ALIGNMENT),
    (dict(T=0, X=None, residual=None, gamma=None, H=None, Y=None, codes=None, scales=None), OK),
])
def test_norm(lib, change, want):
    a = dict(NORM)
    a.update(change)
    assert lib.bcq_rms_norm(*a.values()) == want
