"""The language-model operators of this framework as measured: their cases, a plain form of each in
elementary torch operations, and the calls a user makes.

Kinds of case:
  score    log probabilities of given tokens, entropy and the top alternatives of logit rows
  loss     the same statistics, then their gradient with respect to the logits
  matvec   a few feature rows times 4-bit weights with group scales
  act8     an activation whose input is kept in 8 bits, then its backward (act "none": kept and restored)
  wgrad    the weight gradient of a linear layer from its input kept in 8 bits
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 32                                   # elements that share one scale (MXFP4 weights, 8-bit checkpoints)
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def listed():
    return [
        # one decoded token's logits over the 131k-label head: latency
        dict(name="score_one", kind="score", N=1, V=131072, dtype="f32", pad=0, M=1, k=5, masked=0.0),
        # a batch of queries scored against the 670k-label head, several positive labels each
        dict(name="score_labels", kind="score", N=256, V=670000, dtype="f32", pad=0, M=8, k=5, masked=0.0),
        # a constrained decode: odd vocabulary, rows of a wider buffer, a fifth of the tokens masked out
        dict(name="score_masked", kind="score", N=37, V=100003, dtype="bf16", pad=5, M=1, k=20, masked=0.2),
        # a training step's token loss with its gradient, the largest
        dict(name="loss_large", kind="loss", N=4096, V=131072, dtype="bf16", pad=0, M=1, masked=0.0),
        # a ragged batch in FP32 with several targets a row
        dict(name="loss_odd", kind="loss", N=333, V=32003, dtype="f32", pad=0, M=3, masked=0.1),
        # one query against the 131k-label head in MXFP4
        dict(name="matvec_one", kind="matvec", fmt="mxfp4", N=1, D=768, L=131072, group=32, zeros=False),
        # sixteen queries against the 3M-label head in MXFP4
        dict(name="matvec_3m", kind="matvec", fmt="mxfp4", N=16, D=768, L=3000000, group=32, zeros=False),
        # one token through a layer of integer weights with zero points, odd row count: the smallest
        dict(name="matvec_int4", kind="matvec", fmt="int4", N=1, D=4096, L=4099, group=32, zeros=True),
        # an encoder's wide activation over a batch of tokens
        dict(name="act8_gelu", kind="act8", T=16384, D=4096, dtype="bf16", act="gelu"),
        # a layer input kept and restored, odd token count
        dict(name="act8_keep", kind="act8", T=1537, D=768, dtype="bf16", act="none"),
        # the weight gradient of a wide layer
        dict(name="wgrad_large", kind="wgrad", T=16384, O=2048, D=4096),
        # the weight gradient of an encoder layer from a short, odd batch
        dict(name="wgrad_odd", kind="wgrad", T=1001, O=768, D=768),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["score", "loss", "matvec", "act8", "wgrad"])
    if kind in ("score", "loss"):
        dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
        V = _spread(rng, 1000, 1000000)
        most = (680 << 20) // SIZE[dtype] // V if kind == "score" else (1 << 30) // SIZE[dtype] // V
        c = dict(kind=kind, N=_spread(rng, 1, max(1, min(4096, most))), V=V, dtype=dtype, pad=rng.choice([0, 0, 1, 6, 64]),
                 M=rng.choice([1, 1, 2, 8]), masked=rng.choice([0.0, 0.0, 0.1, 0.5]))
        if kind == "score":
            c["k"] = rng.choice([0, 1, 5, 20, 64])
        return c
    if kind == "matvec":
        fmt = rng.choice(["mxfp4", "int4"])
        D = 256 * _spread(rng, 1, 32) if fmt == "mxfp4" else 128 * _spread(rng, 1, 64)
        return dict(kind=kind, fmt=fmt, N=_spread(rng, 1, 32), D=D, L=_spread(rng, 256, min(3000000, (2 << 30) // D)),
                    group=32 if fmt == "mxfp4" else rng.choice([32, 64, 128]), zeros=fmt == "int4" and rng.random() < 0.5)
    if kind == "act8":
        D = 32 * _spread(rng, 2, 256)
        return dict(kind=kind, T=_spread(rng, 1, (64 << 20) // D), D=D, dtype=rng.choice(["f32", "bf16", "bf16", "f16"]),
                    act=rng.choice(["none", "relu", "silu", "gelu"]))
    O, D = 8 * _spread(rng, 8, 512), 32 * _spread(rng, 2, 128)
    return dict(kind=kind, T=_spread(rng, 1, min(32768, (1 << 37) // (O * D))), O=O, D=D)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    kind = case["kind"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case)
    if kind in ("score", "loss"):
        N, V, M = case["N"], case["V"], case["M"]
        z = normal(N, V + case["pad"]).mul_(3.0)
        if case["masked"]:                   # tokens that a grammar or a filter rules out
            z.masked_fill_(torch.rand((N, V + case["pad"]), generator=g, device=dev) < case["masked"], float("-inf"))
        s["Z"] = z.to(DTYPES[case["dtype"]])[:, :V]
        ids = torch.randint(0, V, (N, M), generator=g, device=dev, dtype=torch.int32)
        if M > 1:                            # rows have different numbers of tokens: negative ids fill the rest
            ids[:, 1:].masked_fill_(torch.rand((N, M - 1), generator=g, device=dev) < 0.3, -1)
        s["ids"] = ids
        s["Z"].scatter_(1, ids.clamp(min=0).long(), 4.0)      # a token that was drawn is allowed and likely
        if kind == "loss":
            s["dlogp"] = normal(N, M)
            s["dentropy"] = torch.full((N,), -0.01, device=dev)
    elif kind == "matvec":
        N, D, L, G = case["N"], case["D"], case["L"], case["group"]
        s["X"] = normal(N, D).to(torch.bfloat16)
        if case["fmt"] == "mxfp4":           # rows of D/2 code bytes, then D/32 scale bytes
            s["W"] = torch.randint(0, 256, (L, 17 * D // 32), generator=g, device=dev, dtype=torch.uint8)
            s["W"][:, D // 2:] = torch.randint(119, 122, (L, D // 32), generator=g, device=dev, dtype=torch.uint8)
            s["scales"] = s["zero"] = None
        else:
            s["W"] = torch.randint(0, 256, (L, D // 2), generator=g, device=dev, dtype=torch.uint8)
            s["scales"] = (torch.rand((L, D // G), generator=g, device=dev) * 0.01 + 0.002).to(torch.bfloat16)
            s["zero"] = (torch.randint(6, 11, (L, D // G), generator=g, device=dev, dtype=torch.uint8)
                         if case["zeros"] else None)
    elif kind == "act8":
        # features of different scales, as an encoder's hidden units have
        x = normal(case["T"], case["D"]) * torch.exp(normal(case["D"]))
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["dy"] = normal(case["T"], case["D"]).mul_(1e-2).to(DTYPES[case["dtype"]])
    else:
        magnitude = torch.randint(0, 127, (case["T"], case["D"]), generator=g, device=dev, dtype=torch.uint8)
        sign = torch.randint(0, 2, (case["T"], case["D"]), generator=g, device=dev, dtype=torch.uint8) * 128
        s["codes"] = magnitude + sign        # E4M3 codes without the NaN ones
        s["scales"] = torch.randint(116, 121, (case["T"], case["D"] // BLOCK), generator=g, device=dev, dtype=torch.uint8)
        s["dy"] = normal(case["T"], case["O"]).mul_(1e-2).to(torch.bfloat16)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import precision_label_chunk_amd as elmo
    kind = s["kind"]
    if kind == "score":
        r = elmo.logprobs(s["Z"], s["ids"], k=s["k"])
        out = dict(logp=r.logp, entropy=r.entropy, row_max=r.row_max, log_sum=r.log_sum)
        if s["k"]:
            out.update(top_idx=r.top_idx, top_logp=r.top_logp)
        return out
    if kind == "loss":
        r = elmo.logprobs(s["Z"], s["ids"])
        dz = elmo.logprobs_backward(s["Z"], s["ids"], r, s["dlogp"], dentropy=s["dentropy"])
        return dict(logp=r.logp, entropy=r.entropy, dz=dz)
    if kind == "matvec":
        fmt = elmo.ELMO_W_MXFP4 if s["fmt"] == "mxfp4" else elmo.ELMO_W_INT4
        return dict(y=elmo.w4_matvec(s["W"], s["X"], wfmt=fmt, scales=s["scales"], zeros=s["zero"]))
    if kind == "act8":
        if s["act"] == "none":
            codes, scales, _ = elmo.ckpt8_save(s["x"])
            return dict(x=elmo.ckpt8_load(codes, scales, dtype=torch.bfloat16))
        codes, scales, y = elmo.ckpt8_save(s["x"], act=s["act"])
        return dict(y=y, dx=elmo.ckpt8_act_grad(s["dy"], codes, scales, act=s["act"]))
    return dict(dw=elmo.ckpt8_weight_grad(s["dy"], s["codes"], s["scales"]))


# ---- plain forms -------------------------------------------------------------------------------
def _plain_stats(s):
    z, ids = s["Z"].float(), s["ids"]
    m = z.max(dim=1).values
    y = z - m[:, None]
    e = torch.exp(y)
    total = e.sum(dim=1)
    logs = torch.log(total)
    entropy = logs - (e * y.clamp(min=-1e4)).sum(dim=1) / total
    given = y.gather(1, ids.clamp(min=0).long()) - logs[:, None]
    logp = torch.where(ids < 0, torch.zeros_like(given), given)
    return z, y, m, logs, entropy, logp


def _plain(s):
    kind = s["kind"]
    if kind == "score":
        z, y, m, logs, entropy, logp = _plain_stats(s)
        out = dict(logp=logp, entropy=entropy, row_max=m, log_sum=logs)
        if s["k"]:
            # order by (logit falling, token rising): one whole number for both
            b = (z + 0.0).view(torch.int32)
            b = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
            place = torch.arange(z.shape[1], device=z.device)
            key = b * (1 << 32) + ((1 << 32) - 1 - place)
            best = key.topk(s["k"], dim=1).values
            idx = (1 << 32) - 1 - (best & 0xFFFFFFFF)
            out.update(top_idx=idx.to(torch.int32), top_logp=y.gather(1, idx) - logs[:, None])
        return out
    if kind == "loss":
        z, y, m, logs, entropy, logp = _plain_stats(s)
        ids = s["ids"]
        given = torch.where(ids < 0, torch.zeros_like(s["dlogp"]), s["dlogp"])
        lp = y - logs[:, None]
        p = torch.exp(lp)
        dz = p * (-given.sum(dim=1)[:, None] - s["dentropy"][:, None] * (lp.clamp(min=-1e4) + entropy[:, None]))
        dz.scatter_add_(1, ids.clamp(min=0).long(), given)
        return dict(logp=logp, entropy=entropy, dz=dz.to(s["Z"].dtype))
    if kind == "matvec":
        D, L, G = s["D"], s["L"], s["group"]
        codes = s["W"][:, :D // 2]
        if s["fmt"] == "mxfp4":
            table = torch.tensor(E2M1, device=codes.device)
            w = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=2).view(L, D // G, G)
            scale = torch.exp2(s["W"][:, D // 2:].float() - 127.0)
        else:
            w = torch.stack([codes & 15, codes >> 4], dim=2).view(L, D // G, G).float()
            w = w - (s["zero"].float()[:, :, None] if s["zero"] is not None else 8.0)
            scale = s["scales"].float()
        w = (w * scale[:, :, None]).view(L, D)
        return dict(y=s["X"].float() @ w.t())
    if kind == "act8":
        x = s["x"].float()
        kept = _plain_keep(x)
        if s["act"] == "none":
            return dict(x=kept.to(torch.bfloat16))
        y, _ = _plain_act(x, s["act"])
        _, d = _plain_act(kept, s["act"])
        return dict(y=y.to(s["x"].dtype), dx=(s["dy"].float() * d).to(s["dy"].dtype))
    T, D = s["codes"].shape
    x = s["codes"].view(torch.float8_e4m3fn).float().view(T, D // BLOCK, BLOCK)
    x = (x * torch.exp2(s["scales"].float() - 127.0)[:, :, None]).view(T, D)
    return dict(dw=s["dy"].float().t() @ x)


def _plain_keep(x):
    """x as its 8-bit form holds it: blocks of 32 share the smallest power of two 2^X with
    max|x| <= 448 2^X, the elements are E4M3 to nearest even."""
    T, D = x.shape
    b = x.view(T, D // BLOCK, BLOCK)
    part, power = torch.frexp(b.abs().amax(dim=2, keepdim=True))          # amax = part 2^power, part in [0.5, 1)
    X = (power - 9 + (part > 0.875).int()).clamp(min=-127)
    return (torch.ldexp(b, -X).to(torch.float8_e4m3fn).float() * torch.exp2(X.float())).view(T, D)


def _plain_act(x, act):
    """act(x) and its derivative."""
    if act == "relu":
        return x.clamp(min=0), (x > 0).float()
    if act == "silu":
        q = 1.0 / (1.0 + torch.exp(-x))
        return x * q, q * (1.0 + x * (1.0 - q))
    c = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return x * c, c + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))


# ---- what one pass cannot do without -----------------------------------------------------------
def work(case):
    kind = case["kind"]
    if kind == "score":
        n = case["N"] * case["V"]
        return dict(bytes=n * SIZE[case["dtype"]] + case["N"] * (8 * case["M"] + 12 + 8 * case["k"]), flops=6 * n)
    if kind == "loss":                       # the gradient needs a row's sum first: the logits are read for each
        n = case["N"] * case["V"]
        return dict(bytes=3 * n * SIZE[case["dtype"]] + case["N"] * (12 * case["M"] + 12), flops=12 * n)
    if kind == "matvec":
        N, D, L = case["N"], case["D"], case["L"]
        groups = D // case["group"]
        per = groups if case["fmt"] == "mxfp4" else groups * (3 if case["zeros"] else 2)
        return dict(bytes=L * (D // 2 + per) + 2 * N * D + 4 * N * L, flops=2 * N * L * D)
    if kind == "act8":
        n, e = case["T"] * case["D"], SIZE[case["dtype"]]
        kept = n + n // BLOCK                # written by the forward, read by the backward
        if case["act"] == "none":
            return dict(bytes=n * e + 2 * kept + 2 * n, flops=4 * n)
        return dict(bytes=2 * n * e + 2 * kept + 2 * n * e, flops=30 * n)
    T, O, D = case["T"], case["O"], case["D"]
    return dict(bytes=2 * T * O + T * D + T * D // BLOCK + 4 * O * D, flops=2 * T * O * D)


# ---- the definitions in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("score", "loss"):
        N, V = s["Z"].shape
        step = max(1, (1 << 27) // V)
        parts = [_exact_rows(s, slice(a, a + step)) for a in range(0, N, step)]
        return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}
    if kind == "matvec":
        D, L = s["D"], s["L"]
        step = max(1, (1 << 28) // D)
        return dict(y=torch.cat([s["X"].double() @ _exact_weights(s, slice(a, a + step)).t() for a in range(0, L, step)], dim=1))
    if kind == "act8":
        x = s["x"].double()
        blocks = x.unflatten(1, (-1, BLOCK))
        top = blocks.abs().amax(dim=2, keepdim=True)
        # the smallest whole X with top <= 448 2^X
        X = torch.ceil(torch.log2(top / 448.0).clamp(min=-127.0))
        X = X + (top > 448.0 * torch.exp2(X)).double()
        X = (X - (top <= 448.0 * torch.exp2(X - 1)).double()).clamp(min=-127.0)
        a = (blocks / torch.exp2(X)).abs()
        # spacing of E4M3 numbers around a: 2^-9 below 2^-6, else an eighth of the power of two below a
        unit = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0**-6))) - 3.0)
        kept = (torch.sign(blocks) * torch.round(a / unit) * unit * torch.exp2(X)).flatten(1)
        if s["act"] == "none":
            return dict(x=kept)
        dy = s["dy"].double()
        if s["act"] == "relu":
            return dict(y=torch.relu(x), dx=torch.where(kept > 0, dy, torch.zeros_like(dy)))
        if s["act"] == "silu":
            q = torch.sigmoid(kept)
            return dict(y=x * torch.sigmoid(x), dx=dy * (q + kept * q * (1 - q)))
        y = 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
        d = 0.5 * torch.erfc(-kept / math.sqrt(2.0)) + kept * torch.exp(-kept.square() / 2) / math.sqrt(2 * math.pi)
        return dict(y=y, dx=dy * d)
    code = s["codes"].int()
    power, part = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(power == 0, part * 2.0**-9, (8.0 + part) * torch.exp2(power.double() - 10.0))
    x = torch.where(code >= 128, -mag, mag) * torch.exp2(s["scales"].double() - 127.0).repeat_interleave(BLOCK, dim=1)
    return dict(dw=s["dy"].double().t().contiguous() @ x)


def _exact_rows(s, rows):
    z, ids = s["Z"][rows].double(), s["ids"][rows].long()
    m = z.amax(dim=1, keepdim=True)
    lse = torch.logsumexp(z, dim=1, keepdim=True)
    lp = z - lse
    p = lp.exp()
    entropy = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(dim=1)
    real = ids >= 0
    logp = torch.where(real, lp.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=torch.float64, device=z.device))
    if s["kind"] == "score":
        out = dict(logp=logp, entropy=entropy, row_max=m[:, 0], log_sum=(lse - m)[:, 0])
        if s["k"]:
            out.update(top_idx=None, top_logp=lp.topk(s["k"], dim=1).values)
        return out
    g = s["dlogp"][rows].double() * real
    dz = -p * g.sum(dim=1, keepdim=True)
    dz.scatter_add_(1, ids.clamp(min=0), g)
    surprise = torch.where(p > 0, lp, torch.zeros_like(lp)) + entropy[:, None]
    dz -= s["dentropy"][rows].double()[:, None] * p * surprise
    return dict(logp=logp, entropy=entropy, dz=dz)


def _exact_weights(s, rows):
    D, G = s["D"], s["group"]
    raw = s["W"][rows]
    byte = raw[:, :D // 2].int()
    c = torch.empty((raw.shape[0], D), dtype=torch.int32, device=raw.device)
    c[:, 0::2], c[:, 1::2] = byte % 16, byte // 16
    if s["fmt"] == "mxfp4":
        mag = c % 8
        val = torch.where(mag < 2, mag.double() / 2, (2 + mag % 2).double() * torch.exp2((mag // 2 - 2).double()))
        val = torch.where(c >= 8, -val, val)
        scale = torch.exp2(raw[:, D // 2:].double() - 127)
        return val * scale.repeat_interleave(G, dim=1)
    zero = s["zero"][rows].double().repeat_interleave(G, dim=1) if s["zero"] is not None else 8.0
    return (c.double() - zero) * s["scales"][rows].double().repeat_interleave(G, dim=1)
