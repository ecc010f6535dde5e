"""Gradients from features where the upstream gradients of the labels and of the log partition lie far apart, and where
their sum in a row leaves binary32's range.

Tolerances: those of the tests of ordinary sizes. G is held in units of which its bound (the largest |dlse| + 2 sum |dlogp| of a
row) is at most 2^60 (FP16: 2^15), so that BF16's smallest numbers, 2^-133, are 2^-193 of the bound; probabilities below 2^-126 count as 0: another 2^-126 of it."""
import pytest
import torch

from test_gpu_linear_logprobs import BF, F32, HALF, HF, LEAST, _case, _gradients, _near, elmo  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(elmo, X, W, ids, up, dlse):  # noqa: F811
    r = elmo.linear_logprobs(X, W, ids)
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, dx=torch.empty(X.shape, device="cuda"),
                                           dw=torch.empty(W.shape, device="cuda"))
    dX, dW, tX, tW = _gradients(X, W, ids, up, dlse)
    most = float((dlse.cpu().double().abs() + 2 * up.cpu().double().abs().sum(1)).max()) * (2.0**-193 + 2.0**-126)
    tX, tW = tX + most * W.cpu().double().abs().sum(0), tW + most * X.cpu().double().abs().sum(0)
    assert float(dX.abs().max()) < 2e38 and float(dW.abs().max()) < 2e38          # (they can be held)
    _near(dx, dX, tX + HALF[F32] * (dX.abs() + tX) + LEAST[F32], "dX")
    _near(dw, dW, tW + 2 * HALF[F32] * (dW.abs() + tW) + 2 * LEAST[F32], "dW")


@pytest.mark.parametrize("N", [20, 200])
@pytest.mark.parametrize("label,partition", [(1e-35, 1e10), (1e-30, 1e9), (1e-20, 1e20), (1e-37, 1e36), (1e-30, 1.0), (1.0, 1e-30)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_labels_and_partition_far_apart(elmo, dtype, label, partition, N):  # noqa: F811
    X, W, ids, up, dlse = _case(N, 2000, 64, 1, dtype, seed=6)
    _check(elmo, X, W, ids, up * label, dlse * partition)


@pytest.mark.parametrize("N", [20, 200])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_of_either_kind(elmo, dtype, N):  # noqa: F811
    """Every second row has the partition's gradient only, the others the labels'."""
    X, W, ids, up, dlse = _case(N, 500, 64, 2, dtype, seed=7)
    up, dlse = up * 1e-32, dlse * 1e9
    up[::2] = 0
    dlse[1::2] = 0
    _check(elmo, X, W, ids, up, dlse)


@pytest.mark.parametrize("N", [20, 200])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_bound_beyond_the_range(elmo, dtype, N):  # noqa: F811
    """The gradients of a row add up to more than binary32 holds; they themselves, and the results, do not."""
    X, W, ids, up, dlse = _case(N, 500, 64, 3, dtype, seed=8)
    X, W = X / 64, W / 8
    up, dlse = -3e38 + 0 * up, 3e38 + 0 * dlse
    up[1::3], dlse[1::3] = up[1::3] * 1e-3, dlse[1::3] * 1e-3
    up[2::3], dlse[2::3] = 0, 0
    ids[:, 1:] = -1
    ids[0, 1] = (ids[0, 0] + 1) % 500
    _check(elmo, X, W, ids, up, dlse)
