"""What the example serves: the 8-bit chain step by step against the same chain in plain operations, and its distance from
the BF16 weights' log probabilities.

The chain is exact up to its last step: codes are whole numbers that 64 bits decide, the sums are whole, a result is one
conversion and two multiplications in binary32; gelu is torch's own on both sides. The log probabilities are a binary32
softmax over V logits: off by at most (64 + 24 + 3 (log2 V + 3) + 8) u, and 8 u of their own size."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
U = 2.0**-24


def _codes(x):
    """The nearest whole numbers to 127 x / max|x| (halves to even; a quotient in 64 bits is a half only where it is one:
    operands of at most 24 bits) and the scales."""
    d = x.double()
    top = d.abs().amax(1, keepdim=True)
    return torch.round(d * 127.0 / top), (top / 127.0).float()


def _product(a, b):
    (x, s), (w, t) = a, b
    return (x @ w.t()).float() * s * t.t()


def _trained(monkeypatch):
    """The example's parameters after a few steps, and what it returns."""
    import feature_softmax as ex
    made = []

    class Kept(ex.Params):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            made.append(self)
    monkeypatch.setattr(ex, "Params", Kept)
    losses, served, exact = ex.main(steps=8)
    x, ids = next(iter(ex.data(1, 16, 128, 1000)))
    return ex, made[0].w, x, ids, served, exact


def test_served_by_the_same_chain(monkeypatch):
    ex, w, x, ids, served, exact = _trained(monkeypatch)
    h = torch.nn.functional.gelu(_product(_codes(x), _codes(w[0]))).to(torch.bfloat16)
    z = _product(_codes(h), _codes(w[1])).double()
    want = torch.log_softmax(z, 1).topk(5, dim=1)
    tol = (64 + 24 + 3 * (math.log2(1000) + 3) + 8) * U + 8 * U * want.values.abs()
    assert bool(((served.top_logp.double() - want.values).abs() <= tol).all())
    assert torch.equal(z.gather(1, served.top_idx.long()), z.gather(1, want.indices))


def test_distance_from_the_bf16_weights(monkeypatch):
    """Half a code of each operand, as in the test of served logits, in both layers. In between, a hidden feature that is off
    by e before gelu (slope below 1.13) is off by 1.13 e behind it; the BF16 side rounds x W^T and both sides round gelu to
    BF16, half a unit, 2^-8, each. If every logit of a row is off by at most B, its k-th largest log probability is off by at
    most 2 B."""
    ex, w, x, ids, served, exact = _trained(monkeypatch)

    def half_codes(a, b):
        s, t = _codes(a)[1].double(), _codes(b)[1].double().t()
        a, b = a.double().abs(), b.double().abs()
        return a.sum(1, keepdim=True) * t / 2 + b.sum(1)[None, :] * s / 2 + a.shape[1] * s * t / 4
    z8, z = _product(_codes(x), _codes(w[0])), (x @ w[0].t()).float()
    h8, h = (torch.nn.functional.gelu(v).to(torch.bfloat16).double() for v in (z8, z))
    e = half_codes(x, w[0]) * (1 + 1e-5) + 2.0**-8 * z.double().abs() * (1 + 2.0**-7) + 1e-6
    off = 1.13 * e + 2.0**-8 * (h8.abs() + h.abs()) + 1e-6
    assert bool(((h8 - h).abs() <= off).all())
    B = ((h8 - h).abs() @ w[1].double().abs().t() + half_codes(h8.to(torch.bfloat16), w[1]) * (1 + 1e-5)).amax(1, keepdim=True) + 1e-4
    assert bool(((served.top_logp.double() - exact.top_logp.double()).abs() <= 2 * B).all())
    plain = (h @ w[1].double().t())
    lp = torch.log_softmax(plain, 1)
    assert bool(((exact.top_logp.double() - lp.topk(5, dim=1).values).abs() < 1e-4).all())
    assert bool(((exact.logp.double() - lp.gather(1, ids.long())).abs() < 1e-4).all())
    # the served labels are as good as the BF16 ones, up to the same distance
    assert bool((lp.gather(1, served.top_idx.long()).amin(1) >= lp.topk(5, dim=1).values[:, 4] - 2 * B[:, 0]).all())
