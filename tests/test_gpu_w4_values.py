"""Products of a few rows with 4-bit weights at the ends of the formats' ranges, for every result type
and over more than one tile per wave, against float64. Tolerances as in test_gpu_w4_matvec.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
# (rows, features, result type): rows in registers, in LDS (one and eight waves to a tile), from the caches
FORMS = [(1, 256, torch.float32), (20, 768, torch.float32), (3, 4096, torch.float32), (32, 4096, torch.bfloat16)]


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("N,D,dtype", FORMS)
@pytest.mark.parametrize("e", [0, 1, 126, 127, 251, 252, 253, 254])
def test_every_code_at_the_ends_of_the_scales(elmo, N, D, dtype, e):
    """Label j holds code j at one feature and zeros elsewhere. Weights below 2^128 come back exactly, down
    to 2^-128 (scale code 0 is 2^-127); the others are infinite, as in binary32."""
    k = D - 37
    W = torch.zeros((16, 17 * D // 32), dtype=torch.uint8)
    W[:, k // 2] = torch.arange(16, dtype=torch.uint8) << (4 * (k & 1))
    W[:, D // 2 + k // 32] = e
    X = torch.zeros((N, D), dtype=torch.bfloat16, device="cuda")
    X[N - 1, k] = 1.0
    y = elmo.w4_matvec(W.cuda(), X, out_dtype=dtype).cpu().double()
    w = (E2M1 * 2.0 ** (e - 127)).float().double()               # (2^128 and more: infinite)
    assert torch.equal(y[N - 1], w)
    rest = torch.where(torch.isinf(w), torch.full_like(w, float("nan")), torch.zeros_like(w))   # 0 w
    assert torch.equal(y[:N - 1].nan_to_num(nan=7.0), rest.nan_to_num(nan=7.0).expand(N - 1, 16))


@pytest.mark.parametrize("N,D,dtype", FORMS)
@pytest.mark.parametrize("inf", [float("inf"), float("-inf")])
def test_infinite_features(elmo, N, D, dtype, inf):
    """One infinite feature: the other rows are untouched. MXFP4: its row is infinite with the weight's
    sign, NaN where the weight is 0. Integer codes: its row is NaN."""
    L, G, k, n = 50, 32, D - 100, N // 2
    g = torch.Generator().manual_seed(D)
    X = torch.randn((N, D), generator=g).to(torch.bfloat16).cuda()
    Xi = X.clone()
    Xi[n, k] = inf
    others = [i for i in range(N) if i != n]
    raw = torch.randint(0, 256, (L, D // 2), generator=g, dtype=torch.uint8)
    raw[:16, k // 2] = torch.arange(16, dtype=torch.uint8) * 17                # every code at the feature
    W = torch.cat([raw, torch.full((L, D // 32), 120, dtype=torch.uint8)], 1).cuda()
    a, b = elmo.w4_matvec(W, X, out_dtype=dtype), elmo.w4_matvec(W, Xi, out_dtype=dtype)
    assert torch.equal(a[others], b[others]) and bool(torch.isfinite(a).all())
    code = (raw[:, k // 2].long() >> (4 * (k & 1))) & 15
    want = inf * E2M1[code]                                                    # (inf times 0: NaN)
    assert torch.equal(b[n].cpu().double().nan_to_num(nan=7.0, posinf=1.0, neginf=-1.0), want.nan_to_num(nan=7.0, posinf=1.0, neginf=-1.0))
    s = torch.full((L, D // G), 0.25, dtype=torch.bfloat16, device="cuda")
    z = torch.randint(0, 16, (L, D // G), generator=g, dtype=torch.uint8).cuda()
    for zeros in (None, z):
        kw = dict(wfmt=elmo.ELMO_W_INT4, scales=s, zeros=zeros, out_dtype=dtype)
        a, b = elmo.w4_matvec(raw.cuda(), X, **kw), elmo.w4_matvec(raw.cuda(), Xi, **kw)
        assert torch.equal(a[others], b[others]) and bool(torch.isfinite(a).all())
        assert bool(b[n].isnan().all())


def _weights(elmo, fmt, L, D, G, seed):
    """(W, arguments, function giving float64 (weights, sizes that the roundings are of) of a slice of labels)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8, device="cuda")

    if fmt == "mx":
        W = draw(0, 256, (L, 17 * D // 32))
        W[:, D // 2:] = draw(117, 123, (L, D // 32))
        table = E2M1.cuda()
    else:
        W, z = draw(0, 256, (L, D // 2)), draw(0, 16, (L, D // G))
        s = (torch.rand((L, D // G), generator=g, device="cuda") * 0.05 - 0.02).to(torch.bfloat16)

    def values(rows):
        r = W[rows]
        c = torch.stack([r[:, :D // 2] & 15, r[:, :D // 2] >> 4], 2).flatten(1).int()
        if fmt == "mx":
            w = table[c] * torch.exp2(r[:, D // 2:].double() - 127).repeat_interleave(32, 1)
            return w, w.abs()
        sc, zp = (t[rows].double().repeat_interleave(G, 1) for t in (s, z))
        return (c.double() - zp) * sc, (c.double() + zp) * sc.abs()

    return W, {} if fmt == "mx" else dict(wfmt=elmo.ELMO_W_INT4, scales=s, zeros=z), values


def _close(y, X, values, eps, unit=0.0, tiny=0.0):
    x = X.double()
    for a in range(0, y.shape[1], 8192):
        rows = slice(a, a + 8192)
        w, size = values(rows)
        ref = x @ w.t().contiguous()
        tol = eps * (x.abs() @ size.t().contiguous()) + unit * ref.abs() + tiny
        off = (y[:, rows].double() - ref).abs()
        assert bool((off <= tol).all()), f"labels from {a}: off by {off.max():.3e}, {(off / tol).max():.3g} of the tolerance"


@pytest.mark.parametrize("dtype,unit,tiny", [(torch.float32, 0.0, 0.0), (torch.bfloat16, 2.0**-8, 2.0**-134),
                                             (torch.float16, 2.0**-11, 2.0**-25)])
@pytest.mark.parametrize("N,D,G", [(3, 768, 64), (3, 1088, 32), (9, 768, 128), (13, 2080, 32), (24, 704, 64), (30, 1536, 128)])
def test_integer_codes_in_every_result_type(elmo, N, D, G, dtype, unit, tiny):
    """One and eight waves to a tile, each way of placing the feature rows; results in a wider buffer."""
    L = 1001
    W, kw, values = _weights(elmo, "int4", L, D, G, N)
    X = torch.randn((N, D), generator=torch.Generator().manual_seed(N)).to(torch.bfloat16).cuda()
    print(f"  int4 N={N} D={D} G={G} {dtype}", flush=True)
    wide = torch.zeros((N, L + 9), dtype=dtype, device="cuda")
    y = elmo.w4_matvec(W, X, out=wide[:, 4:4 + L], **kw)
    _close(y, X, values, (16 + D / 128) * U, unit, tiny)
    assert bool((wide[:, :4] == 0).all()) and bool((wide[:, 4 + L:] == 0).all())


@pytest.mark.parametrize("N", [1, 4, 16, 17, 32])
@pytest.mark.parametrize("fmt,L,D,G", [("mx", 32901, 512, 32), ("mx", 70001, 512, 32), ("mx", 70001, 768, 32), ("mx", 40007, 1024, 32),
                                       ("mx", 100003, 1024, 32), ("mx", 70001, 1280, 32), ("int4", 120001, 160, 32),
                                       ("int4", 120001, 768, 64), ("int4", 70001, 1024, 128)])
def test_several_tiles_per_wave(elmo, N, fmt, L, D, G):
    """More tiles of 16 labels than resident waves: a wave's second and third tiles, the last of them short."""
    W, kw, values = _weights(elmo, fmt, L, D, G, N + D)
    X = torch.randn((N, D), generator=torch.Generator().manual_seed(N)).to(torch.bfloat16).cuda()
    print(f"  {fmt} N={N} L={L} D={D} G={G}", flush=True)
    _close(elmo.w4_matvec(W, X, **kw), X, values, ((D / 32 + 48) if fmt == "mx" else (16 + D / 128)) * U)


@pytest.mark.parametrize("fmt,N,D", [("mx", 1, 768), ("mx", 16, 4096), ("int4", 16, 4096), ("int4", 30, 2080)])
def test_graph_replays(elmo, fmt, N, D):
    """Captured once, replayed with new features and the program's own work in between."""
    W, kw, _ = _weights(elmo, fmt, 3001, D, 32, 5)
    X = torch.randn((N, D), device="cuda").to(torch.bfloat16)
    elmo.w4_matvec(W, X, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = elmo.w4_matvec(W, X, **kw)
    for _ in range(4):
        X.copy_(torch.randn((N, D), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, elmo.w4_matvec(W, X, **kw))
