"""Dropout, log probabilities from features with their gradient, and 8-bit integer products run together as the
example uses them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_runs():
    import feature_softmax as ex
    losses, served, exact = ex.main(steps=8)
    assert losses.shape == (8,) and bool(torch.isfinite(losses).all())
    assert served.top_idx.shape == (16, 5) and bool(((served.top_idx >= 0) & (served.top_idx < 1000)).all())
    assert bool((served.top_logp[:, :-1] >= served.top_logp[:, 1:]).all()) and bool((served.top_logp <= 0).all())
    # rows' log probabilities sum to 1 over all labels: served ones come from finite logits
    assert bool(torch.isfinite(served.entropy).all())


@pytest.mark.parametrize("T,V", [(200, 504), (96, 1000)])
def test_gradients_against_autograd(T, V):
    """The weights' gradients of one batch against autograd in float64 of the same values: the saved activations are
    what the 8 bits hold (straight through), every BF16 tensor what BF16 holds, the dropout's mask the one that the
    operator draws. On the way to dW1 there are roundings to BF16 of the upstream gradient at dkept, dh and dz and
    of G (above 128 rows), each at most 2^-8 relative and of random sign; to dW2 only G's. 4 x 2^-8 of the norm
    bounds their sum."""
    import precision_label_chunk_amd as elmo
    import feature_softmax as ex
    F, H = 128, 256
    p = ex.Params([(H, F), (V, H)])
    (x, ids), = ex.data(1, T, F, V)
    loss, (dw1, dw2) = ex.gradients(p, x, ids, step=3, drop=0.25, pull=0.1)
    z = x @ p.w[0].t()
    kept_x = elmo.ckpt8_load(*elmo.ckpt8_save(x)[:2]).double()
    kept_z = elmo.ckpt8_load(*elmo.ckpt8_save(z)[:2], dtype=torch.float32).double()
    h = elmo.ckpt8_save(z, act="gelu")[2]
    hd = elmo.dropout(h, 0.25, 7, 3).double().requires_grad_()
    mask = elmo.dropout(torch.ones_like(h, dtype=torch.float32), 0.25, 7, 3).double()
    w2 = p.w[1].double().requires_grad_()
    logits = hd @ w2.t()
    lp = torch.log_softmax(logits, dim=1).gather(1, ids.long())
    total = -lp.mean() + 0.1 * torch.logsumexp(logits, dim=1).mean()
    total.backward()
    assert abs(float(loss) + float(lp.detach().mean())) < 1e-5 * (1 + abs(float(loss)))
    kz = kept_z.clone().requires_grad_()
    torch.nn.functional.gelu(kz).backward(hd.grad * mask)
    for name, got, want in (("dW1", dw1, kz.grad.t() @ kept_x), ("dW2", dw2, w2.grad)):
        off = float((got.double() - want).norm() / want.norm())
        print(f"  {name} off by {off:.2e} of its norm", flush=True)
        assert off < 4 * 2.0**-8


def test_served_logits_within_their_codes():
    """A served logit differs from that of the same BF16 operands by half a code of each: with s = max|h| / 127 and
    t = max|w| / 127 of its rows at most sum |h| t / 2 + sum |w| s / 2 + D s t / 4."""
    import precision_label_chunk_amd as elmo
    g = torch.Generator(device="cuda").manual_seed(3)
    for N in (1, 20, 70):
        h = torch.randn((N, 256), generator=g, device="cuda").to(torch.bfloat16)
        w = (torch.randn((1003, 256), generator=g, device="cuda") / 16).to(torch.bfloat16)
        (hc, s), (wc, t) = elmo.i8_quantize(h), elmo.i8_quantize(w)
        y = elmo.i8_matmul(hc, s, wc, t, out_dtype=torch.float32).double()
        h, w, s, t = h.double(), w.double(), s.double()[:, None], t.double()[None, :]
        bound = h.abs().sum(1, keepdim=True) * t / 2 + w.abs().sum(1)[None, :] * s / 2 + 256 * s * t / 4
        assert bool(((y - h @ w.t()).abs() <= bound * (1 + 1e-5)).all())
