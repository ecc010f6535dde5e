"""How exactly the gradient's numbers G are held: as the sum of two 16-bit numbers up to 128 rows, and for results in float32
whatever the number of rows; as one for other results above 128 rows. Tolerances as in the tests of ordinary sizes, with h^2 in the
place of G's half unit h where G is two numbers; what binary32 adds to h^2 stays below 2^-10, so that a number lost, or
found in the wrong place, shows."""
import math

import pytest
import torch

from test_gpu_linear_logprobs import BF, F32, HALF, HF, LEAST, U, _case, _near, _plain, elmo  # noqa: F401

pytestmark = pytest.mark.gpu
EDGE = [1, 64, 127, 128, 129]


def _wanted(X, W, ids, up, dlse, dx_type, dw_type):
    """(dX, its tolerance), (dW, its tolerance) before the last rounding."""
    z, m, lse, lp, E, R = _plain(X, W, ids)
    x, w, i = X.cpu().double(), W.cpu().double(), ids.cpu().long()
    N, V = z.shape
    g, e = torch.where(i < 0, torch.zeros(()).double(), up.cpu().double()), dlse.cpu().double()
    c, big = e - g.sum(1), g.abs().sum(1) + e.abs()
    l = z - lse[:, None]
    p = l.exp()
    G, A = p * c[:, None], p * big[:, None]
    rough = c.abs()[:, None] * p * (R[:, None] + (3 * l.abs() / math.log(2) + 8) * U)
    for j in range(i.shape[1]):
        on = torch.zeros_like(G).scatter_(1, i[:, j:j + 1].clamp(min=0), g[:, j:j + 1])
        G, A = G + on, A + on.abs()
    out = []
    for kind in (dx_type, dw_type):
        h = HALF[X.dtype] ** (2 if N <= 128 or kind == F32 else 1)
        off = h * G.abs() + (rough + 8 * U * A) * (1 + h)
        if X.dtype == HF:
            off = off + 2.0**-25 * 2.0**-13 * 2 * big.max()
        out.append(off)
    return ((G @ w, out[0] @ w.abs() + (V + 64) * U * (G.abs() @ w.abs())),
            (G.t() @ x, out[1].t() @ x.abs() + (N + 64) * U * (G.abs().t() @ x.abs())))


def _check(elmo, N, V, D, M, dtype, dx_type, dw_type, seed, accumulate=False, need_dx=True, need_dw=True, chunk=0):  # noqa: F811
    X, W, ids, up, dlse = _case(N, V, D, M, dtype, seed=seed)
    print(f"  {N} x {V} x {D} {dtype}, dX {dx_type}, dW {dw_type}, chunk {chunk}", flush=True)
    r = elmo.linear_logprobs(X, W, ids)
    dx = torch.full((N, D), 5.0, device="cuda", dtype=dx_type)
    dw = torch.randn((V, D), device="cuda").to(dw_type)
    old = dw.cpu().double() if accumulate else 0.0
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, dx=dx if need_dx else None, dw=dw if need_dw else None, chunk=chunk,
                                           accumulate=accumulate, need_dx=need_dx, need_dw=need_dw)
    (dX, tX), (dW, tW) = _wanted(X, W, ids, up, dlse, dx_type, dw_type)
    if need_dx:
        _near(dx, dX, tX + HALF[dx_type] * (dX.abs() + tX) + LEAST[dx_type], "dX")
    if need_dw:
        dW = dW + old
        _near(dw, dW, tW + 2 * HALF[dw_type] * (dW.abs() + tW) + 2 * LEAST[dw_type], "dW")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("chunk", [0, 256])
@pytest.mark.parametrize("N", EDGE)
def test_float32_results_at_the_edge(elmo, N, chunk, dtype):  # noqa: F811
    _check(elmo, N, 1500, 128, 2, dtype, F32, F32, seed=N, chunk=chunk)


@pytest.mark.parametrize("out", [F32, BF, HF])
@pytest.mark.parametrize("N", EDGE)
def test_accumulated_at_the_edge(elmo, N, out):  # noqa: F811
    for chunk in (0, 256):
        _check(elmo, N, 700, 96, 1, BF, out, out, seed=N + 1, chunk=chunk, accumulate=True)


@pytest.mark.parametrize("dx_type,dw_type", [(F32, F32), (BF, F32), (F32, BF), (HF, F32), (F32, HF), (BF, HF)])
@pytest.mark.parametrize("N,V,D", [(300, 1001, 160), (512, 1000, 256), (1000, 257, 64), (1500, 3001, 96)])
def test_results_of_either_type(elmo, N, V, D, dx_type, dw_type):  # noqa: F811
    """Each result by its own type; runs of rows and of labels, which are summed apart."""
    _check(elmo, N, V, D, 1, BF, dx_type, dw_type, seed=N)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_one_result_alone(elmo, dtype):  # noqa: F811
    for chunk in (0, 512):
        _check(elmo, 700, 1100, 64, 2, dtype, F32, F32, seed=3, need_dx=False, chunk=chunk, accumulate=True)
        _check(elmo, 700, 1100, 64, 2, dtype, F32, F32, seed=4, need_dw=False, chunk=chunk)


def test_more_labels_than_a_piece_holds(elmo):  # noqa: F811
    """4.5M labels, two rows, pieces of 2^22 labels: dW is a sum of two products, in float64 on the device a part of the
    labels at a time. G carries 2^-16, E = D u sum |x w| of a logit twice, and R of the row."""
    N, V, D = 2, 4_500_000, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn((V, D), generator=g, device="cuda").to(BF)
    X = torch.randn((N, D), generator=g, device="cuda").to(BF)
    ids = torch.tensor([[V - 1], [(1 << 22) + 5]], device="cuda", dtype=torch.int32)
    r = elmo.linear_logprobs(X, W, ids)
    _, dw = elmo.linear_logprobs_backward(X, W, ids, r, torch.full((N, 1), -1.0, device="cuda"), need_dx=False,
                                          dw=torch.empty((V, D), device="cuda"))
    x, w = X.double(), W.double()
    z = x @ w.t()
    E = D * U * float((x.abs() @ w.abs().t()).max())
    R = (64 + V / 8192 + 24 + 3 * (math.log2(V) + 3) + 8) * U + 2 * E
    l = z - torch.logsumexp(z, 1)[:, None]
    p = l.exp()
    G = p.scatter_add(1, ids.long(), torch.full((N, 1), -1.0, device="cuda", dtype=torch.float64))
    off = 2.0**-16 * G.abs() + 1.01 * p * (R + (3 * l.abs() / math.log(2) + 16) * U)
    off.scatter_add_(1, ids.long(), torch.full((N, 1), 8 * U, device="cuda", dtype=torch.float64))
    assert R < 2.0**-11 and bool(((dw.double() - G.t() @ x).abs() <= 1.01 * (off.t() @ x.abs()) + 1e-30).all())
