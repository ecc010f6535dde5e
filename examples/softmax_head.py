"""A small softmax classifier trained and served with the language-model operators.

Training keeps every activation that the backward needs in 8 bits (ckpt8_save), takes the loss as
token log probabilities with an entropy bonus (logprobs, logprobs_backward over the logits' own
memory), forms the weight gradients from the 8-bit activations (ckpt8_weight_grad) and the
activation's from its saved input (ckpt8_act_grad), and updates BF16 parameters without FP32 master
copies (kahan_update). Serving packs the head to 4-bit codes with group scales and answers single
rows: w4_matvec, then logprobs with the top alternatives.

    python examples/softmax_head.py
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


def train_step(p: Params, x, ids, lr, entropy_weight=1e-3):
    """One step on a batch; returns the mean negative log probability (a device scalar)."""
    w1, w2 = p.w
    tokens = x.shape[0]
    # forward: the backward needs x, z and h; each is kept in 8 bits and nothing else stays
    x8 = elmo.ckpt8_save(x)[:2]
    z8c, z8s, h = elmo.ckpt8_save(x @ w1.t(), act="gelu")
    h8 = elmo.ckpt8_save(h)[:2]
    logits = h @ w2.t()
    stats = elmo.logprobs(logits, ids)
    # loss = -mean(logp) - entropy_weight mean(H)
    dlogp = torch.full_like(stats.logp, -1.0 / tokens)
    dentropy = torch.full_like(stats.entropy, -entropy_weight / tokens)
    dlogits = elmo.logprobs_backward(logits, ids, stats, dlogp, dentropy=dentropy, out=logits)
    dw2 = elmo.ckpt8_weight_grad(dlogits, *h8)
    dh = dlogits @ w2
    dz = elmo.ckpt8_act_grad(dh, z8c, z8s, act="gelu", out=dh)
    dw1 = elmo.ckpt8_weight_grad(dz, *x8)
    p.update((dw1, dw2), lr)
    return -stats.logp.mean()


def pack_int4(w, group=32):
    """4-bit codes (zero point 8) with one BF16 scale per group of `group` features of a row."""
    rows, features = w.shape
    g = w.float().view(rows, features // group, group)
    scales = (g.abs().amax(dim=2) / 7.0).clamp(min=1e-30).to(torch.bfloat16)
    codes = (torch.round(g / scales.float()[:, :, None]).clamp(-8, 7) + 8).to(torch.uint8).view(rows, features // 2, 2)
    return (codes[:, :, 0] | codes[:, :, 1] << 4).contiguous(), scales


def serve(p: Params, head, x, k=5):
    """The k best labels of each row of x with their log probabilities, by the packed head."""
    codes, scales = head
    h = torch.nn.functional.gelu((x @ p.w[0].t()).float()).to(torch.bfloat16)
    logits = elmo.w4_matvec(codes, h, wfmt=elmo.ELMO_W_INT4, scales=scales)
    return elmo.logprobs(logits, k=k)


def main(steps=200, tokens=512, features=128, hidden=256, labels=1000, lr=2.0):
    p = Params([(hidden, features), (labels, hidden)])
    losses = [train_step(p, x, ids, lr) for x, ids in data(steps, tokens, features, labels)]
    losses = torch.stack(losses).cpu()
    head = pack_int4(p.w[1])
    x, ids = next(iter(data(1, 16, features, labels)))
    served = serve(p, head, x)
    exact = elmo.logprobs(torch.nn.functional.gelu((x @ p.w[0].t()).float()) @ p.w[1].float().t(), ids, k=5)
    agree = (served.top_idx[:, 0] == exact.top_idx[:, 0]).float().mean()
    return losses, served, float(agree)


if __name__ == "__main__":
    losses, served, agree = main()
    print(f"mean negative log probability: first step {losses[0]:.3f}, last {losses[-1]:.3f}")
    print(f"first row's alternatives by the 4-bit head: {served.top_idx[0].tolist()}, log probabilities "
          f"{[round(v, 3) for v in served.top_logp[0].tolist()]}")
    print(f"rows whose best label the 4-bit head shares with the BF16 head: {agree:.0%}")
