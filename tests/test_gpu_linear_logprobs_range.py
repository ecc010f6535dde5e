"""Log probabilities from features and their gradients for logits far from zero, up to 2^101.

Every logit is exact in binary32, in any order of its sum: 16 features give +-2^m, the others whole multiples below 2^10 of
2^max(m - 23, 0). Labels come several times over, so that rows have ties (from 2^31 on a spacing of binary32 is 256, and
ties are all there is). With the logits exact, what is left of the other tests' tolerances is R, the exponentials' and
the sum's roundings, and those of the gradient's numbers G; binary32 has no normal numbers below 2^-126, and the exponential gives 0
there: an element of G is off by another |c| 2^-125, for at most half of the exponent's last unit, below 2^24, comes back as a factor of
at most 2^(1/2)."""
import math

import pytest
import torch

from test_gpu_linear_logprobs import BF, F32, HALF, HF, LEAST, U, _near, elmo  # noqa: F401

pytestmark = pytest.mark.gpu
MAGNITUDES = {BF: [0, 22, 23, 24, 25, 28, 30, 31, 32, 33, 35, 66, 101], HF: [0, 22, 23, 24, 25, 28, 30, 31, 32, 33]}
CASES = [(t, m) for t in (BF, HF) for m in [None, *MAGNITUDES[t]]]


def _case(N, V, M, dtype, m, seed=0, D=64):
    """Rows of magnitude 2^m (None: one after the other), every second row negative; m = 0: whole numbers below 2^10."""
    g = torch.Generator().manual_seed(seed)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g).double()
    ms = MAGNITUDES[dtype] if m is None else [m]
    at = torch.tensor([ms[n // 2 % len(ms)] for n in range(N)], dtype=torch.float64)
    X, W = whole(N, D), whole(V // 3 + 1, D)[torch.randint(0, V // 3 + 1, (V,), generator=g)]
    X *= torch.exp2((at - 23).clamp(min=0))[:, None]
    top = 30 if dtype == BF else 14
    X[:, :16] = torch.where(at > 0, torch.exp2(at - 4 - top), torch.zeros(()).double())[:, None]
    X[1::2, :16] *= -1
    W[:, :16] = 2.0**top
    for t in (X, W):
        assert torch.equal(t.to(dtype).double(), t)
    z = X @ W.t()
    assert torch.equal(z.float().double(), z) and float(z.abs().max()) < 2.0**126
    ids = torch.randint(0, V, (N, M), generator=g, dtype=torch.int32)
    ids[:, 0] = z.argmax(1).int()
    ids[::3, 0] = torch.randint(0, V, (len(ids[::3]),), generator=g, dtype=torch.int32)
    up, dlse = torch.randn((N, M), generator=g), torch.randn((N,), generator=g)
    return X.to(dtype).cuda(), W.to(dtype).cuda(), ids.cuda(), up.cuda(), dlse.cuda(), z


def _check(elmo, N, V, M, dtype, m, seed=0):  # noqa: F811
    X, W, ids, up, dlse, z = _case(N, V, M, dtype, m, seed)
    print(f"  {N} x {V}, M={M} {dtype}, 2^{m}", flush=True)
    r = elmo.linear_logprobs(X, W, ids)
    i, x, w = ids.cpu().long(), X.cpu().double(), W.cpu().double()
    top = z.max(1).values
    d = z - top[:, None]
    logs = torch.logsumexp(d, 1)
    R = (64 + V / 8192 + 24 + 3 * (math.log2(V) + 3) + 8) * U
    lp = d.gather(1, i) - logs[:, None]
    assert torch.equal(r.row_max.cpu().double(), top)
    _near(r.log_sum, logs, R + 4 * U * logs, "log_sum")
    _near(r.logp, lp, R + 8 * U * lp.abs(), "logp")
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, dx=torch.empty(X.shape, device="cuda"),
                                           dw=torch.empty(W.shape, device="cuda"))
    g, e = up.cpu().double(), dlse.cpu().double()
    c, big = e - g.sum(1), g.abs().sum(1) + e.abs()
    l = d - logs[:, None]
    p = l.exp()
    G, A = p * c[:, None], p * big[:, None]
    rough = c.abs()[:, None] * (p * (R + (3 * l.abs() / math.log(2) + 8) * U) + 2.0**-125)
    for j in range(ids.shape[1]):
        on = torch.zeros_like(G).scatter_(1, i[:, j:j + 1], g[:, j:j + 1])
        G, A = G + on, A + on.abs()
    h = HALF[dtype] ** (2 if N <= 128 else 1)
    off = h * G.abs() + (rough + 8 * U * A) * (1 + h)
    if dtype == HF:
        off = off + 2.0**-25 * 2.0**-13 * 2 * big.max()
    for got, ref, tol, K, name in ((dx, G @ w, off @ w.abs(), (G.abs() @ w.abs()) * (V + 64), "dX"),
                                   (dw, G.t() @ x, off.t() @ x.abs(), (G.abs().t() @ x.abs()) * (N + 64), "dW")):
        tol = tol + U * K
        _near(got, ref, tol + 2 * HALF[F32] * (ref.abs() + tol) + 2 * LEAST[F32], name)


@pytest.mark.parametrize("dtype,m", CASES)
def test_one_magnitude(elmo, dtype, m):  # noqa: F811
    """m = None: rows of every magnitude next to each other."""
    _check(elmo, 40, 700, 2, dtype, m, seed=1)


@pytest.mark.parametrize("dtype,m", [(BF, None), (HF, None), (BF, 33), (HF, 33)])
@pytest.mark.parametrize("N,V", [(300, 5003), (129, 300), (2000, 9001), (1, 1)])
def test_tile_shapes(elmo, N, V, dtype, m):  # noqa: F811
    _check(elmo, N, V, 1, dtype, m, seed=2)


def test_rows_near_zero_keep_their_bits(elmo):  # noqa: F811
    """A row's results do not depend on the magnitude of its neighbours."""
    X, W, ids, up, dlse, _ = _case(300, 1000, 2, BF, 0, seed=3)
    far = _case(300, 1000, 2, BF, None, seed=3)[0]
    Y = X.clone()
    Y[::2] = far[::2]
    W[:, :16] = 2.0**30
    X[:, :16] = 0
    Y[1::2] = X[1::2]
    r, s = elmo.linear_logprobs(X, W, ids), elmo.linear_logprobs(Y, W, ids)
    for a, b in zip(r, s):
        assert torch.equal(a[1::2], b[1::2])
    dx, dy = (elmo.linear_logprobs_backward(x, W, ids, t, up, dlse=dlse, need_dw=False)[0] for x, t in ((X, r), (Y, s)))
    assert torch.equal(dx[1::2], dy[1::2]) and bool(dy.isfinite().all())
