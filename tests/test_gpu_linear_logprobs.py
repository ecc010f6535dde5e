"""Log probabilities straight from features and weights, and their gradients, against a plain float64
implementation on the CPU.

Tolerances (u = 2^-24). A logit is a binary32 sum of D exact products: off by at most E = D u sum |x w|, with the
largest E of a row for its maximum. A row's sum of exponentials adds at most V non-negative terms in
parts of 64 and a tree, at most c = 64 + V / 8192 + 24 additions deep; each term carries 3 (|y| + 1) u of its
exponent and the exponential's 2 u (as for the operator on given logits: weighted by the terms the mean of |y| is at
most log2 V + 2), so log s is off by R = (c + 3 (log2 V + 3) + 8) u + 2 E.
Gradient: G = c p + g carries p's R + (3 |y| + 8) u + 2 E relative and a few roundings of c and g (8 u of |c| p +
sum |g|), then half a unit h of its own type (h^2 up to 128 rows, where a second number of the type holds what the first
leaves); dX and dW are binary32 sums of exact products of it, off by at most
K u sum |G W|, and round once to their type: half a unit relative, and for FP16 results at least 2^-25, half the
spacing 2^-24 of its numbers below 2^-14."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
LEAST = {F32: 2.0**-150, BF: 2.0**-134, HF: 2.0**-25}      # half the spacing of a type's smallest numbers


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def _pitched(t, pad):
    """t as rows of a wider buffer."""
    if not pad:
        return t.cuda()
    return torch.cat([t, torch.full((t.shape[0], pad), 7.0, dtype=t.dtype)], 1).cuda()[:, :t.shape[1]]


def _case(N, V, D, M, dtype, seed=0, pad=0, far=4.0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn((V, D), generator=g) * (1.5 / math.sqrt(D))).to(dtype)
    ids = torch.randint(0, V, (N, M), generator=g, dtype=torch.int32)
    x = torch.randn((N, D), generator=g)
    if M:
        x += W[ids[:, 0].long()].float() * (torch.rand((N, 1), generator=g) * far)
    if M > 1:
        ids[:, 1:][torch.rand((N, M - 1), generator=g) < 0.3] = -1
        ids[0, 1] = ids[0, 0]                # the same label twice
    up = torch.randn((N, M), generator=g)
    dlse = torch.randn((N,), generator=g)
    return _pitched(x.to(dtype), pad), _pitched(W, pad), ids.cuda(), up.cuda(), dlse.cuda()


def _plain(X, W, ids):
    x, w = X.cpu().double(), W.cpu().double()
    z = x @ w.t()
    m = z.max(1).values
    lse = torch.logsumexp(z, 1)
    i = ids.cpu().long()
    lp = z.gather(1, i.clamp(min=0)) - lse[:, None] if i.numel() else torch.zeros(i.shape, dtype=torch.float64)
    size = x.abs() @ w.abs().t()
    V, D = w.shape
    E = D * U * size.max(1).values
    R = (64 + V / 8192 + 24 + 3 * (math.log2(V) + 3) + 8) * U + 2 * E
    return z, m, lse, torch.where(i < 0, torch.zeros_like(lp), lp), E, R


def _near(got, ref, tol, what):
    got = got.cpu().double()
    off = (got - ref).abs()
    assert got.isfinite().all(), what
    assert bool((off <= tol).all()), f"{what}: off by {off.max():.3e}, {(off / tol).nan_to_num().max():.3g} of the tolerance"


def _check_forward(elmo, X, W, ids):
    print(f"  linear_logprobs {tuple(X.shape)} {tuple(W.shape)} {X.dtype} M={ids.shape[1]}", flush=True)
    r = elmo.linear_logprobs(X, W, ids)
    z, m, lse, lp, E, R = _plain(X, W, ids)
    _near(r.row_max, m, E + U * m.abs(), "row_max")
    _near(r.log_sum, lse - m, R + E + 4 * U * (lse - m).abs(), "log_sum")
    _near(r.logp, lp, (R + 2 * E)[:, None] + 8 * U * lp.abs(), "logp")
    return r


def _gradients(X, W, ids, up, dlse):
    """float64 (dX, dW) and their tolerances before the last rounding, for G held with half unit `h`."""
    z, m, lse, lp, E, R = _plain(X, W, ids)
    x, w, i = X.cpu().double(), W.cpu().double(), ids.cpu().long()
    N, V = z.shape
    g = torch.where(i < 0, torch.zeros((), dtype=torch.float64), up.cpu().double())
    c = -g.sum(1) if dlse is None else dlse.cpu().double() - g.sum(1)
    big = g.abs().sum(1) + (0 if dlse is None else dlse.cpu().double().abs())
    y = (z - lse[:, None]) / math.log(2)
    p = (z - lse[:, None]).exp()
    G = p * c[:, None]
    A = p * big[:, None]
    rough = c.abs()[:, None] * p * (R[:, None] + (3 * y.abs() + 8) * U)
    for j in range(i.shape[1]):
        on = torch.zeros_like(G)
        on.scatter_(1, i[:, j:j + 1].clamp(min=0), g[:, j:j + 1])
        G, A = G + on, A + on.abs()
    h = HALF[X.dtype] ** (2 if N <= 128 else 1)
    off = h * G.abs() + (rough + 8 * U * A) * (1 + h)
    if X.dtype == HF:                        # below its normal numbers FP16 is off by 2^-25 of the scaled value
        off = off + 2.0**-25 * 2.0**-13 * 2 * big.max()
    dX, dW = G @ w, G.t() @ x
    tX = off @ w.abs() + (V + 64) * U * (G.abs() @ w.abs())
    tW = off.t() @ x.abs() + (N + 64) * U * (G.abs().t() @ x.abs())
    return dX, dW, tX, tW


def _check_backward(elmo, X, W, ids, up, dlse, r=None, **kw):
    r = r or elmo.linear_logprobs(X, W, ids)
    old = kw["dw"].cpu().double() if kw.get("accumulate") else 0.0
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, **kw)
    dX, dW, tX, tW = _gradients(X, W, ids, up, dlse)
    if dx is not None:
        _near(dx, dX, tX + HALF[dx.dtype] * (dX.abs() + tX) + LEAST[dx.dtype], "dX")
    if dw is not None:
        dW = dW + old
        _near(dw, dW, tW + 2 * HALF[dw.dtype] * (dW.abs() + tW) + 2 * LEAST[dw.dtype], "dW")
    return dx, dw


SHAPES = [(1, 1, 32, 1), (1, 257, 64, 1), (2, 128, 32, 0), (3, 255, 96, 2), (31, 1000, 64, 1), (64, 129, 160, 3), (65, 513, 256, 1),
          (255, 300, 32, 2), (257, 256, 128, 1), (300, 4097, 96, 8), (513, 769, 288, 1)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,V,D,M", SHAPES)
def test_sizes(elmo, N, V, D, M, dtype):
    X, W, ids, up, dlse = _case(N, V, D, M, dtype, seed=N + V)
    r = _check_forward(elmo, X, W, ids)
    _check_backward(elmo, X, W, ids, up, dlse, r)


@pytest.mark.parametrize("N,V,D", [(1, 131072, 768), (5, 70001, 1024), (4096, 300, 64), (2000, 5003, 512), (700, 1000, 2048)])
def test_long(elmo, N, V, D):
    """Many label tiles, many tokens, many features; runs of tokens and labels that are summed apart."""
    X, W, ids, up, dlse = _case(N, V, D, 1, BF, seed=7)
    r = _check_forward(elmo, X, W, ids)
    _check_backward(elmo, X, W, ids, up, None, r)


@pytest.mark.parametrize("pad", [8, 24])
def test_pitches(elmo, pad):
    X, W, ids, up, dlse = _case(77, 600, 96, 2, BF, pad=pad)
    assert X.stride(0) == 96 + pad
    r = _check_forward(elmo, X, W, ids)
    dx = torch.full((77, 96 + pad), 3.0, device="cuda")
    dw = torch.full((600, 96 + pad), 3.0, device="cuda", dtype=HF)
    _check_backward(elmo, X, W, ids, up, dlse, r, dx=dx[:, :96], dw=dw[:, :96])
    assert bool((dx[:, 96:] == 3).all()) and bool((dw[:, 96:] == 3).all())


@pytest.mark.parametrize("chunk", [1, 256, 700, 5000])
def test_pieces(elmo, chunk):
    """Any number of pieces, the last one shorter."""
    X, W, ids, up, dlse = _case(130, 1500, 128, 3, BF, seed=3)
    _check_backward(elmo, X, W, ids, up, dlse, chunk=chunk, dx=torch.empty((130, 128), device="cuda"),
                    dw=torch.empty((1500, 128), device="cuda"))


@pytest.mark.parametrize("out", [F32, BF, HF])
def test_accumulate(elmo, out):
    X, W, ids, up, dlse = _case(600, 700, 64, 1, BF, seed=4)
    for chunk in (0, 256):
        dw = torch.randn((700, 64), device="cuda").to(out)
        _check_backward(elmo, X, W, ids, up, dlse, dw=dw, accumulate=True, need_dx=False, chunk=chunk)


def test_one_gradient_alone(elmo):
    X, W, ids, up, dlse = _case(40, 700, 96, 1, HF, seed=5)
    r = elmo.linear_logprobs(X, W, ids)
    both = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse)
    dx, none = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, need_dw=False)
    assert none is None
    none, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, need_dx=False)
    assert none is None
    _check_backward(elmo, X, W, ids, up, dlse, r, need_dx=False)
    _check_backward(elmo, X, W, ids, up, dlse, r, need_dw=False)
    assert both[0].shape == dx.shape and both[1].shape == dw.shape


@pytest.mark.parametrize("scale", [1e-12, 1e-6, 1.0, 1e6])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sizes_of_the_upstream_gradient(elmo, dtype, scale):
    """Nothing is lost to FP16's range: G is scaled by the gradients given."""
    X, W, ids, up, dlse = _case(50, 2000, 64, 1, dtype, seed=6)
    _check_backward(elmo, X, W, ids, up * scale, dlse * scale, dx=torch.empty((50, 64), device="cuda"),
                    dw=torch.empty((2000, 64), device="cuda"))
    _check_backward(elmo, X, W, ids, up * 0, dlse * scale, dx=torch.empty((50, 64), device="cuda"),
                    dw=torch.empty((2000, 64), device="cuda"))


def test_zero_upstream(elmo):
    X, W, ids, up, _ = _case(20, 500, 64, 1, BF)
    r = elmo.linear_logprobs(X, W, ids)
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up * 0)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


def test_confident_rows(elmo):
    """Rows whose given label has nearly all the probability: 1 - p keeps its digits."""
    X, W, ids, up, dlse = _case(64, 1000, 64, 1, BF, seed=8, far=10.0)
    r = _check_forward(elmo, X, W, ids)
    assert float(r.logp.max()) > -1e-3
    _check_backward(elmo, X, W, ids, -up.abs(), None, r, dx=torch.empty((64, 64), device="cuda"),
                    dw=torch.empty((1000, 64), device="cuda"))


@pytest.mark.parametrize("factor", [30.0, 3000.0])
def test_large_logits(elmo, factor):
    """Logits far from zero, of both signs: the row's maximum is taken off before the exponential."""
    X, W, ids, up, dlse = _case(40, 700, 64, 2, BF, seed=9)
    X = (X.float() * factor).to(BF)
    _check_forward(elmo, X, W, ids)
    _check_forward(elmo, X, (W.float() * 0 - 0.05).to(BF), ids)


def test_no_label_and_unknown_labels(elmo):
    X, W, ids, up, dlse = _case(6, 300, 64, 2, BF, seed=10)
    ids[0] = -1
    ids[1] = torch.tensor([-5, 299], device="cuda", dtype=torch.int32)
    _check_forward(elmo, X, W, ids)
    _check_backward(elmo, X, W, ids, up, dlse)
    ids[2, 0] = 300
    r = elmo.linear_logprobs(X, W, ids)
    assert bool(r.logp[2, 0].isnan()) and int(r.logp.isnan().sum()) == 1
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse)
    assert bool(dx[2].isnan().all()) and int(dx.isnan().any(1).sum()) == 1


def test_values_out_of_range_stay_in_their_row(elmo):
    """A NaN feature makes its own row NaN, the other rows keep their bits; a NaN weight row enters every sum."""
    X, W, ids, up, dlse = _case(300, 700, 64, 1, BF, seed=11)
    r = elmo.linear_logprobs(X, W, ids)
    dx, _ = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse)
    Y = X.clone()
    Y[299, 5] = float("nan")
    s = elmo.linear_logprobs(Y, W, ids)
    assert bool(s.logp[299].isnan().all()) and bool(s.log_sum[299].isnan())
    assert torch.equal(s.logp[:299], r.logp[:299]) and torch.equal(s.row_max[:299], r.row_max[:299])
    dy, dw = elmo.linear_logprobs_backward(Y, W, ids, s, up, dlse=dlse)
    assert bool(dy[299].isnan().all()) and torch.equal(dy[:299], dx[:299]) and bool(dw.isnan().all())
    bad = up.clone()
    bad[17] = float("nan")
    dy, _ = elmo.linear_logprobs_backward(X, W, ids, r, bad, dlse=dlse)
    keep = torch.arange(300, device="cuda") != 17
    assert bool(dy[17].isnan().all()) and bool(dy[keep].isfinite().all())


def test_empty_rows_and_infinities(elmo):
    """A row of nothing but -inf logits has no gradient; +inf makes its row NaN."""
    X = torch.ones((4, 32), device="cuda", dtype=BF)
    W = torch.zeros((300, 32), device="cuda", dtype=BF)
    W[:, 0] = 1.0
    X[1, 0] = float("-inf")
    X[2, 0] = float("inf")
    X[:, 1:] = 0.0
    ids = torch.tensor([[3], [4], [5], [-1]], device="cuda", dtype=torch.int32)
    W[:, 1:] = 1.0                           # (no 0 x inf)
    r = elmo.linear_logprobs(X, W, ids)
    assert r.row_max[1] == -math.inf and r.log_sum[1] == 0 and r.logp[1, 0] == -math.inf
    assert bool(r.logp[2].isnan()) and bool(r.log_sum[2].isnan()) and r.logp[3, 0] == 0
    assert abs(float(r.logp[0, 0]) + math.log(300)) < 1e-5
    dx, _ = elmo.linear_logprobs_backward(X, W, ids, r, torch.ones((4, 1), device="cuda"), dlse=torch.ones(4, device="cuda"))
    assert bool((dx[1] == 0).all()) and bool(dx[2].isnan().all()) and bool(dx[0].isfinite().all()) and bool(dx[3].isfinite().all())


def test_no_rows(elmo):
    X, W = torch.empty((0, 64), device="cuda", dtype=BF), torch.ones((50, 64), device="cuda", dtype=BF)
    ids = torch.empty((0, 1), device="cuda", dtype=torch.int32)
    r = elmo.linear_logprobs(X, W, ids)
    assert r.logp.shape == (0, 1)
    dw = torch.ones((50, 64), device="cuda")
    up = torch.empty((0, 1), device="cuda")
    elmo.linear_logprobs_backward(X, W, ids, r, up, dw=dw, accumulate=True)
    assert bool((dw == 1).all())
    elmo.linear_logprobs_backward(X, W, ids, r, up, dw=dw)
    assert bool((dw == 0).all())


def test_differences(elmo):
    """The gradient against differences of the forward itself, in directions of X and W that bfloat16 holds."""
    X, W, ids, up, dlse = _case(16, 400, 64, 2, BF, seed=12)
    r = elmo.linear_logprobs(X, W, ids)
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, dx=torch.empty((16, 64), device="cuda"),
                                           dw=torch.empty((400, 64), device="cuda"))

    def value(x, w):
        s = elmo.linear_logprobs(x, w, ids)
        real = (ids >= 0)
        return float((s.logp.double() * up.double() * real).sum() + ((s.row_max.double() + s.log_sum.double()) * dlse.double()).sum())
    # steps of 2^-4 keep X + step exact where |X| < 16 has it; second-order errors cancel in the difference of
    # both sides, third-order ones are about step^2 / 6 of the gradient's size: 2^-8, and G's half unit as much
    for t, d in ((X, dx), (W, dw)):
        g = torch.Generator(device="cuda").manual_seed(1)
        for _ in range(3):
            n, k = (int(torch.randint(0, s, (1,), generator=g, device="cuda")) for s in t.shape)
            old = t[n, k].clone()
            hi, lo = (old + 2.0**-4).clone(), (old - 2.0**-4).clone()
            v = []
            for s in (hi, lo):
                t[n, k] = s
                v.append(value(X, W))
            t[n, k] = old
            want = (v[0] - v[1]) / float(hi - lo)
            size = float(d.abs().max())
            assert abs(float(d[n, k]) - want) < 0.02 * size + 1e-3


def test_repeats_and_workspaces(elmo):
    """The same bits every time, in a workspace of any content, one used twice among them."""
    X, W, ids, up, dlse = _case(300, 3000, 96, 2, BF, seed=13)
    first = elmo.linear_logprobs(X, W, ids)
    need = elmo.lib().elmo_linear_logprobs_backward_workspace_bytes(300, 3000, 96, 2, 0, 1, 1)
    grads = elmo.linear_logprobs_backward(X, W, ids, first, up, dlse=dlse)
    for fill in (0, 255, 85):
        ws = torch.full((max(need, 1 << 22),), fill, device="cuda", dtype=torch.uint8)
        r = elmo.linear_logprobs(X, W, ids, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(r, first))
        assert all(torch.equal(a, b) for a, b in zip(elmo.linear_logprobs_backward(X, W, ids, r, up, dlse=dlse, workspace=ws), grads))


def test_graph_and_streams(elmo):
    """Recorded and replayed on new inputs, with eager work between; two streams at once."""
    X, W, ids, up, dlse = _case(100, 2000, 64, 1, BF, seed=14)
    other = _case(100, 2000, 64, 1, BF, seed=15)

    def step(a):
        r = elmo.linear_logprobs(a[0], a[1], a[2])
        return (*r, *elmo.linear_logprobs_backward(a[0], a[1], a[2], r, a[3], dlse=a[4], chunk=512))
    mine = [t.clone() for t in (X, W, ids, up, dlse)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(mine)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(mine)
    for a in ((X, W, ids, up, dlse), other, (X, W, ids, up, dlse)):
        for t, s in zip(mine, a):
            t.copy_(s)
        want = step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    want = [step((X, W, ids, up, dlse)), step(other)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st, a in zip(streams, ((X, W, ids, up, dlse), other)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(step(a))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_refusals(elmo):
    X, W, ids, up, dlse = _case(4, 40, 64, 1, BF)
    r = elmo.linear_logprobs(X, W, ids)
    with pytest.raises(ValueError):
        elmo.linear_logprobs(X, W.to(HF), ids)
    with pytest.raises(ValueError):
        elmo.linear_logprobs(X, W[:, :32], ids)
    with pytest.raises(ValueError):
        elmo.linear_logprobs(X, W, ids.long())
    with pytest.raises(ValueError):
        elmo.linear_logprobs(X, W, ids.cpu())
    with pytest.raises(elmo.ElmoError):
        elmo.linear_logprobs(X.float(), W.float(), ids)
    with pytest.raises(elmo.ElmoError):
        elmo.linear_logprobs(X[:, :48].contiguous(), W[:, :48].contiguous(), ids)
    with pytest.raises(elmo.ElmoError):      # rows that are not 16-byte aligned
        elmo.linear_logprobs(torch.empty((4, 68), device="cuda", dtype=BF)[:, :64], W, ids)
    with pytest.raises(ValueError):
        elmo.linear_logprobs_backward(X, W, ids, r, None)
    with pytest.raises(ValueError):
        elmo.linear_logprobs_backward(X, W, ids, r, up, accumulate=True)
    with pytest.raises(ValueError):
        elmo.linear_logprobs_backward(X, W, ids, r, up, need_dx=False, need_dw=False)
    with pytest.raises(ValueError):
        elmo.linear_logprobs_backward(X, W, ids, r, up, dw=torch.empty((40, 32), device="cuda"))
    with pytest.raises(elmo.ElmoError):
        elmo.linear_logprobs_backward(X, W, ids, r, up, chunk=-1)
