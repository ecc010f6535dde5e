"""Products of a few rows with 4-bit weights at the ends of the formats' ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu
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
