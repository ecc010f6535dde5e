"""Token log probabilities over rows long enough that every wave streams many chunks (16 to 40 each):
sums rescaled, thresholds carried and shared again from chunk to chunk; the gradient's main loop, and
its smallest values. Every row against float64 on the GPU; tolerances as in test_gpu_logprobs.py."""
import math

import pytest
import torch

from test_gpu_logprobs import TINY, TYPES, U, UNIT, _R

pytestmark = pytest.mark.gpu
KINDS = 12


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def _logits(N, V, dtype, seed):
    """Rows of twelve kinds in turn: random, rising, falling, a rising bound with noise, ties of a few values,
    all equal, masked but for one in a thousand, masked but for a few at the end, masked by the lowest
    value, runs that favour one wave, a large magnitude, few large among many small."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    low = torch.finfo(dtype).min
    at = torch.arange(V, device="cuda", dtype=torch.float32)
    Z = torch.empty((N, V), dtype=dtype, device="cuda")
    for n in range(N):
        kind, noise = n % KINDS, torch.randn(V, generator=g, device="cuda")
        if kind == 0:
            z = 3 * noise
        elif kind == 1:
            z = at * (20.0 / V)
        elif kind == 2:
            z = -at * (20.0 / V)
        elif kind == 3:
            z = at * (8.0 / V) + noise
        elif kind == 4:
            z = torch.floor(noise.clamp(-2, 2))
        elif kind == 5:
            z = torch.full_like(noise, float(n % 7) - 3)
        elif kind == 6:
            z = torch.where(torch.rand(V, generator=g, device="cuda") < 0.999, torch.full_like(noise, -math.inf), noise)
        elif kind == 7:
            z = torch.where(at < V - 70, torch.full_like(noise, -math.inf), noise)
        elif kind == 8:
            z = torch.where(torch.rand(V, generator=g, device="cuda") < 0.9, torch.full_like(noise, low), noise)
        elif kind == 9:
            z = torch.where((at * (16.0 / V)).floor() == n // KINDS % 16, 5 + noise, noise)
        elif kind == 10:
            z = 300 * noise
        else:
            z = torch.where(torch.rand(V, generator=g, device="cuda") < 1e-4, 10 + noise, 0.1 * noise)
        Z[n] = z.clamp(min=low).to(dtype) if kind == 8 else z.to(dtype)
    return Z


def _ids(N, V, M, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    ids = torch.randint(0, V, (N, M), generator=g, dtype=torch.int32, device="cuda")
    ids[:, 1:][torch.rand((N, M - 1), generator=g, device="cuda") < 0.3] = -1
    return ids


def _within(got, ref, tol, what, n0):
    got = got.double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    off = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(same | (off <= tol))
    assert not bool(bad.any()), f"{what}: row {n0 + int(bad.nonzero()[0, 0])}, off by {off.max():.3e}"


def _stats(z):
    """float64 rows -> (m, log s, log p, entropy); no empty rows here."""
    m = z.amax(1, keepdim=True)
    y = z - m
    e = y.exp()
    s = e.sum(1, keepdim=True)
    H = s.log() - torch.where(e > 0, e * y, torch.zeros_like(e)).sum(1, keepdim=True) / s
    return m[:, 0], s.log()[:, 0], y - s.log(), H[:, 0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V", [(1040, 130001), (256, 600007)])       # one block per row, and four
def test_many_chunks_per_wave(elmo, N, V, dtype):
    Z, ids = _logits(N, V, dtype, V), _ids(N, V, 3, V)
    runs = {k: elmo.logprobs(Z, ids, k=k) for k in (0, 1, 5, 20, 64)}
    print(f"  logprobs {N} x {V} {dtype}", flush=True)
    R = _R(V)
    for a in range(0, N, 64):
        r = slice(a, min(N, a + 64))
        z = Z[r].double() + 0.0
        m, logs, lp, H = _stats(z)
        i = ids[r].long()
        given = torch.where(i < 0, torch.zeros((), dtype=torch.float64, device="cuda"), lp.gather(1, i.clamp(min=0)))
        order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :64]
        best = lp.gather(1, order)
        for k, o in runs.items():
            _within(o.row_max[r], m, 0.0, "row_max", a)
            _within(o.log_sum[r], logs, R, "log_sum", a)
            _within(o.entropy[r], H, R * (2 + H) + 4 * U * H, "entropy", a)
            _within(o.logp[r], given, R + 4 * U * given.abs(), "logp", a)
            if k:
                wrong = (o.top_idx[r].long() != order[:, :k]).any(1).nonzero()
                assert wrong.numel() == 0, f"k = {k}: row {a + int(wrong[0])}"
                _within(o.top_logp[r], best[:, :k], R + 4 * U * best[:, :k].abs(), "top_logp", a)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V", [(1040, 130001), (33000, 10007), (3, 8600003)])
def test_gradient_of_many_vectors_per_block(elmo, N, V, dtype):
    """(33000 rows: a block per row; 8.6M tokens: the most blocks per row, thousands of vectors each)"""
    if N > 2000:
        Z = torch.randn((N, V), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).mul_(3).to(dtype)
    else:
        Z = _logits(N, V, dtype, V + 1)
    ids = _ids(N, V, 2, V)
    g = torch.Generator(device="cuda").manual_seed(9)
    dlogp, dh = torch.randn((N, 2), generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    print(f"  grad {N} x {V} {dtype}", flush=True)
    stats = elmo.logprobs(Z, ids)
    got = elmo.logprobs_backward(Z, ids, stats, dlogp, dentropy=dh)
    plain = elmo.logprobs_backward(Z, ids, stats, dlogp)
    rows = max(1, (1 << 23) // V)
    for a in range(0, N, rows):
        r = slice(a, min(N, a + rows))
        _, _, lp, H = _stats(Z[r].double())
        p, i = lp.exp(), ids[r].long()
        up = torch.where(i < 0, torch.zeros((), dtype=torch.float64, device="cuda"), dlogp[r].double())
        hot = torch.zeros_like(lp).scatter_add_(1, i.clamp(min=0), up)
        size0 = p * up.abs().sum(1, keepdim=True) + torch.zeros_like(lp).scatter_add_(1, i.clamp(min=0), up.abs())
        surprise = torch.where(p > 0, lp, torch.zeros_like(lp))
        for out, e in ((plain, torch.zeros_like(dh[r].double()[:, None])), (got, dh[r].double()[:, None])):
            ref = p * (-up.sum(1, keepdim=True) - e * (surprise + H[:, None])) + hot
            size = size0 + p * e.abs() * (surprise.abs() + H[:, None])
            spread = p * surprise.abs() * (size / p.clamp(min=1e-300)).clamp(max=1e30)
            tol = 2 * (_R(V) + 14 * U) * size + 5 * U * spread + UNIT[dtype] * ref.abs() + TINY[dtype]
            _within(out[r], ref, tol, "dZ", a)
    assert torch.equal(elmo.logprobs_backward(Z, ids, stats, dlogp, dentropy=dh, out=Z), got)   # in place


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1999, 2000])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_of_small_probabilities(elmo, dtype, V, entropy):
    """Probabilities from 1 down to e^-120 under upstream gradients of a thousand: the products that the
    result's type holds are there, also where the probability alone is below binary32's normal range."""
    Z = (torch.arange(V, device="cuda") * (-120.0 / V)).to(dtype).repeat(2, 1)
    ids = torch.tensor([[0], [V - 1]], dtype=torch.int32, device="cuda")
    dlogp, dh = torch.tensor([[1000.0], [-1000.0]], device="cuda"), torch.tensor([300.0, -300.0], device="cuda")
    got = elmo.logprobs_backward(Z, ids, elmo.logprobs(Z, ids), dlogp, dentropy=dh if entropy else None)
    _, _, lp, H = _stats(Z.double())
    p, e = lp.exp(), (dh if entropy else 0 * dh).double()[:, None]
    hot = torch.zeros_like(lp).scatter_(1, ids.long(), dlogp.double())
    ref = p * (-dlogp.double() - e * (lp + H[:, None])) + hot
    size = p * (1000.0 + e.abs() * (lp.abs() + H[:, None])) + hot.abs()
    tol = (2 * (_R(V) + 13 * U) + 5 * U * lp.abs()) * size + UNIT[dtype] * ref.abs() + TINY[dtype]
    _within(got, ref, tol, "dZ", 0)
    if dtype != torch.float16:
        assert bool((got[ref.abs() > 2.0**-125] != 0).all())
