"""Gradients from features for upstream gradients of zero and at the ends of binary32's range, and where dX needs no sum.

Tolerances of the gradients: those of the tests of ordinary sizes. FP16 holds G scaled by a power of two of at most 2^126, so
that each element is off by a further 2^-25 2^-126 at most, half the spacing of FP16's smallest numbers."""
import pytest
import torch

from test_gpu_linear_logprobs import BF, F32, HALF, HF, LEAST, _case, _gradients, _near, elmo  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [20, 200])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_zero_upstream_of_either_kind(elmo, dtype, N):  # noqa: F811
    """A batch that its mask leaves empty: weights of zero, no labels, no gradient at all."""
    X, W, ids, up, dlse = _case(N, 500, 64, 1, dtype)
    r = elmo.linear_logprobs(X, W, ids)
    none = torch.full_like(ids, -1)
    for i, u, d in ((ids, up * 0, None), (ids, up * 0, dlse * 0), (none, up, None), (none, up, dlse * 0)):
        dx, dw = elmo.linear_logprobs_backward(X, W, i, r, u, dlse=d)
        assert bool((dx == 0).all()) and bool((dw == 0).all())
    r0 = elmo.linear_logprobs(X, W)
    dx, dw = elmo.linear_logprobs_backward(X, W, None, r0, None, dlse=dlse * 0)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("scale", [1e-37, 1e-35, 1e-31, 1e31, 1e36])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_upstream_at_the_ends_of_the_range(elmo, dtype, scale):  # noqa: F811
    X, W, ids, up, dlse = _case(50, 2000, 64, 1, dtype, seed=6)
    r = elmo.linear_logprobs(X, W, ids)
    for u, d in ((up * scale, None), (up * 0, dlse * scale), (up * scale, dlse * scale)):
        dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, u, dlse=d, dx=torch.empty((50, 64), device="cuda"),
                                               dw=torch.empty((2000, 64), device="cuda"))
        dX, dW, tX, tW = _gradients(X, W, ids, u, d)
        if dtype == HF:
            tX, tW = tX + 2.0**-151 * W.cpu().double().abs().sum(0), tW + 2.0**-151 * X.cpu().double().abs().sum(0)
        _near(dx, dX, tX + HALF[F32] * (dX.abs() + tX) + LEAST[F32], "dX")
        _near(dw, dW, tW + 2 * HALF[F32] * (dW.abs() + tW) + 2 * LEAST[F32], "dW")


@pytest.mark.parametrize("out", [F32, BF, HF])
@pytest.mark.parametrize("N,V,D", [(129, 31, 32), (200, 500, 512), (701, 1116, 1216), (4096, 4096, 4096)])
def test_dx_of_one_run(elmo, N, V, D, out):  # noqa: F811
    """Few labels for the rows: dX comes from one run over them, straight to its place, in rows of a wider buffer."""
    X, W, ids, up, dlse = _case(N, V, D, 1, BF, seed=N)
    r = elmo.linear_logprobs(X, W, ids)
    buf = torch.full((N + 1, D + 16), 7.0, device="cuda", dtype=out)
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, dx=buf[:N, :D])
    dX, dW, tX, tW = _gradients(X, W, ids, up, dlse)
    _near(dx, dX, tX + HALF[out] * (dX.abs() + tX) + LEAST[out], "dX")
    _near(dw, dW, tW + 2 * HALF[BF] * (dW.abs() + tW) + 2 * LEAST[BF], "dW")
    assert bool((buf[:N, D:] == 7.0).all()) and bool((buf[N] == 7.0).all())
