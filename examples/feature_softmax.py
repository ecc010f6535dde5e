"""A softmax classifier whose logits never exist: trained straight from features, served in 8-bit integers.

Training: the hidden layer keeps its input and activation input in 8 bits (ckpt8_save), dropout draws its mask
from a counter and draws it again for the backward (dropout, dropout_backward), the loss comes from features
and head weights (linear_logprobs) and its gradients a piece of the vocabulary at a time
(linear_logprobs_backward), BF16 parameters are updated without FP32 copies (kahan_update). Serving: weights
quantised once, each row when it comes (i8_quantize), their product (i8_matmul), the best labels with their
log probabilities (logprobs).

    python examples/feature_softmax.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_label_chunk_amd as elmo  # noqa: E402


def data(steps, tokens, features, labels, seed=0):
    """Batches (x BF16, ids) whose label is a fixed random function of x."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher = torch.randn((features, labels), generator=g, device="cuda")
    for _ in range(steps):
        x = torch.randn((tokens, features), generator=g, device="cuda")
        yield x.to(torch.bfloat16), (x @ teacher).argmax(dim=1, keepdim=True).to(torch.int32)


class Params:
    """BF16 weights with their Kahan compensations."""

    def __init__(self, shapes, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w = [(torch.randn(s, generator=g, device="cuda") / s[1] ** 0.5).to(torch.bfloat16) for s in shapes]
        self.c = [torch.zeros(s, dtype=torch.int16, device="cuda") for s in shapes]

    def update(self, grads, lr):
        for w, c, g in zip(self.w, self.c, grads):
            elmo.kahan_update(w.view(torch.int16), c, g, lr)


def gradients(p: Params, x, ids, step, drop=0.1, seed=7, pull=1e-4):
    """(mean negative log probability, gradients of the weights in FP32) of one batch. The loss adds `pull`
    times the mean of the log partition."""
    w1, w2 = p.w
    tokens = x.shape[0]
    x8 = elmo.ckpt8_save(x)[:2]
    z8c, z8s, h = elmo.ckpt8_save(x @ w1.t(), act="gelu")
    kept = elmo.dropout(h, drop, seed, step, out=h)
    stats = elmo.linear_logprobs(kept, w2, ids)
    dlogp = torch.full_like(stats.logp, -1.0 / tokens)
    dlse = torch.full_like(stats.log_sum, pull / tokens)
    dkept, dw2 = elmo.linear_logprobs_backward(kept, w2, ids, stats, dlogp, dlse=dlse,
                                               dw=torch.empty(w2.shape, dtype=torch.float32, device=w2.device))
    dh = elmo.dropout_backward(dkept, drop, seed, step, out=dkept)
    dz = elmo.ckpt8_act_grad(dh, z8c, z8s, act="gelu", out=dh)
    dw1 = elmo.ckpt8_weight_grad(dz, *x8)
    return -stats.logp.mean(), (dw1, dw2)


def quantised(p: Params):
    """The weights as 8-bit rows with a scale each, made once for serving."""
    return [elmo.i8_quantize(w) for w in p.w]


def serve(weights, x, k=5):
    """The k best labels of each row of x with their log probabilities."""
    z = elmo.i8_matmul(*elmo.i8_quantize(x), *weights[0], out_dtype=torch.float32)
    h = torch.nn.functional.gelu(z).to(torch.bfloat16)
    return elmo.logprobs(elmo.i8_matmul(*elmo.i8_quantize(h), *weights[1], out_dtype=torch.float32), k=k)


def main(steps=200, tokens=512, features=128, hidden=256, labels=1000, lr=2.0):
    p = Params([(hidden, features), (labels, hidden)])
    losses = []
    for step, (x, ids) in enumerate(data(steps, tokens, features, labels)):
        loss, grads = gradients(p, x, ids, step)
        p.update(grads, lr)
        losses.append(loss)
    x, ids = next(iter(data(1, 16, features, labels)))
    served = serve(quantised(p), x)
    h = torch.nn.functional.gelu((x @ p.w[0].t()).float()).to(torch.bfloat16)
    exact = elmo.logprobs(h.float() @ p.w[1].float().t(), ids, k=5)
    return torch.stack(losses).cpu(), served, exact


if __name__ == "__main__":
    losses, served, exact = main()
    agree = (served.top_idx[:, 0] == exact.top_idx[:, 0]).float().mean()
    print(f"mean negative log probability: first step {losses[0]:.3f}, last {losses[-1]:.3f}")
    print(f"first row's alternatives by the 8-bit weights: {served.top_idx[0].tolist()}, log probabilities "
          f"{[round(v, 3) for v in served.top_logp[0].tolist()]}")
    print(f"rows whose best label the 8-bit weights share with the BF16 ones: {agree:.0%}")
