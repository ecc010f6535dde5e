"""The language-model operators run together: the example trains a softmax classifier with 8-bit
checkpoints, its gradients agree with float64 automatic differentiation of the same step, and the
packed head serves what the trained one does."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_learns_and_serves():
    import softmax_head
    losses, served, agree = softmax_head.main()
    print(f"  loss {losses[0]:.3f} -> {losses[-1]:.3f}, agreement {agree:.2f}", flush=True)
    assert bool(torch.isfinite(losses).all())
    # 1000 labels: the first steps are near log 1000 = 6.9; labels follow x, so that the loss falls
    assert losses[0] > 6.0 and losses[-20:].mean() < losses[:5].mean() - 2.0
    assert agree >= 0.7
    assert bool((served.top_logp[:, :-1] >= served.top_logp[:, 1:]).all()) and bool((served.top_logp <= 0).all())


def test_step_gradients_against_autograd():
    """The step's two weight gradients against autograd in float64 of the same values: the saved
    activations are what the 8 bits hold (straight through), every BF16 tensor what BF16 holds.
    Each of the roughly five roundings to BF16 on the way (z, h, logits' gradient, dh, dz) is 2^-9
    relative, the 8-bit roundings of x and h (2^-4 at most, random) enter dW directly and are part of
    the compared values; 3% of the gradient's norm bounds what is left."""
    import precision_label_chunk_amd as elmo
    import softmax_head
    T, F, H, V = 200, 128, 256, 504
    p = softmax_head.Params([(H, F), (V, H)])
    w1, w2 = (w.clone().double() for w in p.w)
    (x, ids), = softmax_head.data(1, T, F, V)
    grads = []
    p.update = lambda g, lr: grads.extend(g)
    softmax_head.train_step(p, x, ids, 0.0, entropy_weight=0.3)
    kept_x = elmo.ckpt8_load(*elmo.ckpt8_save(x)[:2]).double()
    z = (x @ p.w[0].t())
    kept_z = elmo.ckpt8_load(*elmo.ckpt8_save(z)[:2], dtype=torch.float32).double()
    h = elmo.ckpt8_save(z, act="gelu")[2]
    kept_h = elmo.ckpt8_load(*elmo.ckpt8_save(h)[:2]).double()
    logits = (h @ p.w[1].t()).double().requires_grad_()
    lp = torch.log_softmax(logits, dim=1)
    loss = -lp.gather(1, ids.long()).mean() + 0.3 * (lp.exp() * lp).sum(1).mean()
    loss.backward()
    dw2 = logits.grad.t() @ kept_h
    kz = kept_z.clone().requires_grad_()
    torch.nn.functional.gelu(kz).backward(logits.grad @ w2)
    dw1 = kz.grad.t() @ kept_x
    for got, want in zip(grads, (dw1, dw2)):
        off = (got.double() - want).norm() / want.norm()
        print(f"  gradient off by {off:.2e} of its norm", flush=True)
        assert off < 0.03
