"""Operators for a large softmax head and the layers in front of it, as measured: their cases, a plain
form of each in elementary torch operations, and the calls a user makes.

Kinds of case:
  score    log probabilities of given labels straight from features and head weights, no logits kept
  loss     the same, then the gradients of features and weights
  i8       rows quantised to 8-bit integers, then their product with 8-bit weights, both with scales
  dropout  dropout (with a residual added, or none) and its gradient, the mask drawn from a counter
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one query's label probability under the 131k-label head: latency
        dict(name="score_one", kind="score", N=1, V=131072, D=768, dtype="bf16", M=1),
        # an evaluation batch over the 670k-label head, several positive labels each, odd row count
        dict(name="score_labels", kind="score", N=1001, V=670000, D=768, dtype="bf16", M=8),
        # a training step's loss over the 131k-label head, the largest
        dict(name="loss_large", kind="loss", N=4096, V=131072, D=768, dtype="bf16", M=1),
        # a ragged batch in FP16, an odd vocabulary, several targets a row
        dict(name="loss_odd", kind="loss", N=333, V=32003, D=1024, dtype="f16", M=3),
        # the step of the example's classifier
        dict(name="loss_small", kind="loss", N=512, V=1000, D=256, dtype="bf16", M=1),
        # one token through a layer, odd row count
        dict(name="i8_one", kind="i8", N=1, L=4099, D=4096, dtype="bf16", out="bf16"),
        # sixteen queries against the 3M-label head
        dict(name="i8_3m", kind="i8", N=16, L=3000000, D=768, dtype="bf16", out="f32"),
        # a layer over a large batch of tokens
        dict(name="i8_large", kind="i8", N=16384, L=4096, D=4096, dtype="bf16", out="bf16"),
        # a ragged batch against an odd head, features no multiple of 128
        dict(name="i8_odd", kind="i8", N=333, L=32003, D=704, dtype="f16", out="f16"),
        # an encoder's block output over a batch of tokens, added to the residual
        dict(name="dropout_large", kind="dropout", T=16384, D=4096, dtype="bf16", p=0.1, residual=True),
        # odd rows in FP32, half of the features dropped
        dict(name="dropout_odd", kind="dropout", T=1537, D=769, dtype="f32", p=0.5, residual=False),
        # the features of a small batch in front of the head: the smallest
        dict(name="dropout_small", kind="dropout", T=32, D=768, dtype="bf16", p=0.1, residual=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["score", "loss", "loss", "i8", "i8", "dropout"])
    if kind in ("score", "loss"):
        D = 64 * _spread(rng, 1, 32)
        V = _spread(rng, 1000, min(700000, (1 << 29) // D))
        most = min(4096, (1 << 29) // V, 4096 * 131072 * 768 // (V * D))
        return dict(kind=kind, N=_spread(rng, 1, most), V=V, D=D, dtype=rng.choice(["bf16", "bf16", "f16"]),
                    M=rng.choice([1, 1, 2, 8]))
    if kind == "i8":
        D = 64 * _spread(rng, 1, 128)
        L = _spread(rng, 256, min(3000000, (1 << 31) // D))
        most = min(16384, (1 << 27) // L, (1 << 38) // (L * D))
        return dict(kind=kind, N=_spread(rng, 1, most), L=L, D=D, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    out=rng.choice(["bf16", "f16", "f32"]))
    D = _spread(rng, 1, 8192)
    return dict(kind=kind, T=_spread(rng, 1, min(65536, (1 << 26) // D)), D=D, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                p=rng.choice([0.05, 0.1, 0.3, 0.5]), residual=rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    kind = case["kind"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev)

    s = dict(case)
    if kind in ("score", "loss"):
        N, V, D, M = case["N"], case["V"], case["D"], case["M"]
        dtype = DTYPES[case["dtype"]]
        s["W"] = normal(V, D, dtype=dtype).mul_(1.5 / math.sqrt(D))
        ids = torch.randint(0, V, (N, M), generator=g, device=dev, dtype=torch.int32)
        # features point at their first label, some far and some hardly: rows are learned to different degrees
        toward = s["W"][ids[:, 0].long()].float() * (uniform(N, 1) * 8.0)
        s["X"] = (normal(N, D) + toward).to(dtype)
        if M > 1:                            # rows have different numbers of labels: negative ids fill the rest
            ids[:, 1:].masked_fill_(uniform(N, M - 1) < 0.3, -1)
        s["ids"] = ids
        if kind == "loss":                   # the mean over rows, a few of them padding, and a small pull on the partition
            real = (uniform(N) >= 0.05).float()
            s["dlogp"] = (-real / N)[:, None].expand(N, M).contiguous()
            s["dlse"] = real * (1e-3 / N)
    elif kind == "i8":
        N, L, D = case["N"], case["L"], case["D"]
        # features of different scales, as a layer's inputs have
        s["X"] = (normal(N, D) * torch.exp(0.5 * normal(D))).to(DTYPES[case["dtype"]])
        s["W"] = normal(L, D, dtype=torch.float16).mul_(36.0).round_().clamp_(-127.0, 127.0).to(torch.int8)
        s["w_scales"] = (0.5 + uniform(L)) * (0.03 / math.sqrt(D))
    else:
        T, D = case["T"], case["D"]
        dtype = DTYPES[case["dtype"]]
        s["x"], s["dy"] = normal(T, D).to(dtype), normal(T, D).mul_(1e-2).to(dtype)
        s["residual"] = normal(T, D).to(dtype) if case["residual"] else None
        s["seed"], s["step"] = 1000003 * seed + 17, seed % 100000
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import precision_label_chunk_amd as elmo
    kind = s["kind"]
    if kind in ("score", "loss"):
        r = elmo.linear_logprobs(s["X"], s["W"], s["ids"])
        out = dict(logp=r.logp, row_max=r.row_max, log_sum=r.log_sum)
        if kind == "loss":
            out["dx"], out["dw"] = elmo.linear_logprobs_backward(s["X"], s["W"], s["ids"], r, s["dlogp"], dlse=s["dlse"])
        return out
    if kind == "i8":
        codes, scales = elmo.i8_quantize(s["X"])
        return dict(scales=scales, y=elmo.i8_matmul(codes, scales, s["W"], s["w_scales"], out_dtype=DTYPES[s["out"]]))
    y = elmo.dropout(s["x"], s["p"], s["seed"], s["step"], residual=s["residual"])
    return dict(y=y, dx=elmo.dropout_backward(s["dy"], s["p"], s["seed"], s["step"]))


# ---- plain forms -------------------------------------------------------------------------------
def _plain(s):
    kind = s["kind"]
    if kind in ("score", "loss"):
        x, w, ids = s["X"].float(), s["W"].float(), s["ids"]
        z = x @ w.t()
        m = z.max(dim=1).values
        z.sub_(m[:, None])
        given = z.gather(1, ids.clamp(min=0).long())
        e = torch.exp(z)
        logs = torch.log(e.sum(dim=1))
        logp = torch.where(ids < 0, torch.zeros_like(given), given - logs[:, None])
        out = dict(logp=logp, row_max=m, log_sum=logs)
        if kind == "loss":
            up = torch.where(ids < 0, torch.zeros_like(s["dlogp"]), s["dlogp"])
            c = s["dlse"] - up.sum(dim=1)
            dz = e.mul_((c * torch.exp(-logs))[:, None])
            dz.scatter_add_(1, ids.clamp(min=0).long(), up)
            out["dx"], out["dw"] = (dz @ w).to(s["X"].dtype), (dz.t() @ x).to(s["W"].dtype)
        return out
    if kind == "i8":
        # whole codes next to a border: the quotient in 64 bits
        x = s["X"].double()
        top = x.abs().amax(dim=1, keepdim=True)
        codes = torch.round(x * 127.0 / torch.where(top > 0, top, torch.ones_like(top))).float()
        scales = (top[:, 0] / 127.0).float()
        y = (codes @ s["W"].float().t()) * scales[:, None] * s["w_scales"][None, :]
        return dict(scales=scales, y=y.to(DTYPES[s["out"]]))
    T, D = s["x"].shape
    limit = int(math.floor(s["p"] * 65536.0 + 0.5))
    keep = (_plain_draws(T * D, s["seed"], s["step"]).view(T, D) >= limit)
    factor = 65536.0 / (65536.0 - limit)
    y = torch.where(keep, s["x"].float() * factor, torch.zeros((), device=keep.device))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dx = torch.where(keep, s["dy"].float() * factor, torch.zeros((), device=keep.device))
    return dict(y=y.to(s["x"].dtype), dx=dx.to(s["x"].dtype))


def _plain_draws(n, seed, step):
    """The 16 random bits of elements 0 .. n - 1: Philox4x32-10 with key `seed` and counter (i >> 3, step);
    element i takes half (i & 1) of output word (i >> 1) & 3."""
    low = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, device="cuda")
    a, b = block & low, block >> 32
    c, d = torch.full_like(a, step & low), torch.full_like(a, step >> 32)
    k0, k1 = seed & low, (seed >> 32) & low
    for i in range(10):                      # (64-bit products wrap; their halves are right all the same)
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32 & low) ^ b ^ k0, q & low, (p >> 32 & low) ^ d ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([a, b, c, d], dim=1)
    return torch.stack([words & 0xFFFF, words >> 16], dim=2).flatten()[:n]


# ---- what one pass cannot do without -----------------------------------------------------------
def work(case):
    kind = case["kind"]
    if kind in ("score", "loss"):
        N, V, D, M = case["N"], case["V"], case["D"], case["M"]
        operands, rows = 2 * (N + V) * D, N * (8 * M + 8)
        if kind == "score":
            return dict(bytes=operands + rows, flops=2 * N * V * D)
        return dict(bytes=2 * operands + rows + N * (4 * M + 4), flops=6 * N * V * D)
    if kind == "i8":
        N, L, D = case["N"], case["L"], case["D"]
        return dict(bytes=N * D * SIZE[case["dtype"]] + L * D + 4 * L + 4 * N + N * L * SIZE[case["out"]], flops=2 * N * L * D)
    n = case["T"] * case["D"] * SIZE[case["dtype"]]
    return dict(bytes=n * (5 if case["residual"] else 4), flops=12 * case["T"] * case["D"])


# ---- the definitions in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("score", "loss"):
        return _exact_softmax(s)
    if kind == "i8":
        x = s["X"].double()
        top = x.abs().max(dim=1, keepdim=True)[0]
        near = torch.floor(127.0 * x / top.masked_fill(top == 0, 1.0))
        # to the nearest whole number, halves to the even one; the products are whole in 64 bits
        past = 254.0 * x - (2.0 * near + 1.0) * top
        codes = torch.where((past > 0) | ((past == 0) & (near % 2 != 0) & (top > 0)), near + 1, near)
        scales = top / 127.0
        step = max(1, (1 << 28) // max(s["D"], s["N"]))
        y = [(codes @ s["W"][a:a + step].double().t()) * scales * s["w_scales"][a:a + step].double() for a in range(0, s["L"], step)]
        return dict(scales=scales[:, 0], y=torch.cat(y, dim=1))
    T, D = s["x"].shape
    limit = round(s["p"] * 65536)
    kept = torch.from_numpy(_exact_draws(T * D, s["seed"], s["step"]) >= limit).view(T, D).cuda()
    factor = 1.0 / (1.0 - limit / 65536)
    y, dx = s["x"].double() * kept * factor, s["dy"].double() * kept * factor
    return dict(y=y if s["residual"] is None else y + s["residual"].double(), dx=dx)


def _exact_draws(n, seed, step):
    blocks = np.arange(-(-n // 8), dtype=np.uint64)
    mask, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [blocks & mask, blocks >> half, np.full_like(blocks, step % 2**32), np.full_like(blocks, step // 2**32)]
    for turn in range(10):
        key = [np.uint64((seed + turn * 0x9E3779B9) % 2**32), np.uint64((seed // 2**32 + turn * 0xBB67AE85) % 2**32)]
        first, third = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(third >> half) ^ x[1] ^ key[0], third & mask, (first >> half) ^ x[3] ^ key[1], first & mask]
    return np.stack(x, axis=1).astype("<u4").view("<u2").reshape(-1)[:n].astype(np.int32)


def _exact_softmax(s):
    X, W, ids = s["X"].double(), s["W"], s["ids"].long()
    N, V = s["N"], s["V"]
    step = max(1, (1 << 28) // max(N, s["D"]))
    starts = range(0, V, step)
    row_max = torch.full((N,), -math.inf, dtype=torch.float64, device=X.device)
    lse = row_max.clone()
    at = torch.zeros(ids.shape, dtype=torch.float64, device=X.device)
    for a in starts:
        z = X @ W[a:a + step].double().t()
        row_max = torch.maximum(row_max, z.amax(dim=1))
        lse = torch.logaddexp(lse, torch.logsumexp(z, dim=1))
        here = (ids >= a) & (ids < a + z.shape[1])
        at = torch.where(here, z.gather(1, (ids - a).clamp(0, z.shape[1] - 1)), at)
    real = ids >= 0
    out = dict(logp=torch.where(real, at - lse[:, None], torch.zeros_like(at)), row_max=row_max, log_sum=lse - row_max)
    if s["kind"] == "score":
        return out
    up = s["dlogp"].double() * real
    pull = s["dlse"].double() - up.sum(dim=1)
    dx, dw = torch.zeros_like(X), []
    for a in starts:
        w = W[a:a + step].double()
        dz = torch.exp(X @ w.t() - lse[:, None]) * pull[:, None]
        here = (ids >= a) & (ids < a + w.shape[0])
        dz.scatter_add_(1, (ids - a).clamp(0, w.shape[0] - 1), up * here)
        dx += dz @ w
        dw.append(dz.t() @ X)
    return dict(out, dx=dx, dw=torch.cat(dw))
