"""Products of a few BF16 feature rows with 4-bit weights against float64 on the CPU.

Tolerance (u = 2^-24): every product is exact in binary32 (MXFP4: 2 and 8 significant bits; integer
codes: 4 and 8), so only the sums round. A result is a sum of D terms added in some order: off by at
most D u sum|x w|; in matrix products of 32 terms, a block of waves and the join the longest chain of
roundings is shorter, D / 32 products and at most 32 + 16 further additions, so (D / 32 + 48) u
sum|x w| bounds it. With integer codes the terms summed are x c and x z before the scale:
(12 + D / 128) u sum|x| (c + z) s for the block sums (chains of 4 products of 32 terms, the zero
point's and the scale's fma) and the join."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def _codes(raw):
    """[L, bytes] uint8 -> [L, 2 bytes] codes, low nibble first."""
    raw = raw.cpu().long()
    return torch.stack([raw & 15, raw >> 4], 2).flatten(1)


def _mx(L, D, seed, lo=117, hi=123):
    g = torch.Generator().manual_seed(seed)
    W = torch.randint(0, 256, (L, 17 * D // 32), generator=g, dtype=torch.uint8)
    W[:, D // 2:] = torch.randint(lo, hi, (L, D // 32), generator=g, dtype=torch.uint8)
    return W.cuda()


def _mx_values(W, D):
    W = W.cpu()
    return E2M1[_codes(W[:, :D // 2])] * torch.exp2(W[:, D // 2:].double() - 127).repeat_interleave(32, 1)


def _x(N, D, seed, pitch=0):
    g = torch.Generator().manual_seed(seed + 7)
    return torch.randn((N, D + pitch), generator=g).to(torch.bfloat16).cuda()[:, :D]


def _int4(L, D, G, seed, zeros):
    g = torch.Generator().manual_seed(seed)
    W = torch.randint(0, 256, (L, D // 2), generator=g, dtype=torch.uint8).cuda()
    s = (torch.rand((L, D // G), generator=g) * 0.05 - 0.02).to(torch.bfloat16).cuda()
    z = torch.randint(0, 16, (L, D // G), generator=g, dtype=torch.uint8).cuda() if zeros else None
    return W, s, z


def _check(y, ref, tol, unit=0.0):
    y = y.cpu().double()
    off = (y - ref).abs()
    tol = tol + unit * ref.abs()
    assert bool((off <= tol).all()), f"off by {off.max():.3e}, {(off / tol.clamp(min=1e-300)).max():.3g} of the tolerance"


@pytest.mark.parametrize("N", [1, 2, 5, 16, 17, 32])
@pytest.mark.parametrize("L,D", [(1, 256), (15, 512), (17, 768), (1000, 256), (4099, 1024), (333, 4096), (130, 8192),
                                 (70001, 256), (9, 65536)])
def test_mxfp4(elmo, N, L, D):
    W, X = _mx(L, D, L + N), _x(N, D, N)
    print(f"  mxfp4 N={N} L={L} D={D}", flush=True)
    y = elmo.w4_matvec(W, X)
    w, x = _mx_values(W, D), X.cpu().double()
    _check(y, x @ w.t(), (D / 32 + 48) * U * (x.abs() @ w.abs().t()))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N", [1, 4, 5, 16, 17, 32])
@pytest.mark.parametrize("L,D,G", [(1, 32, 32), (15, 96, 32), (17, 128, 128), (1000, 320, 64), (4099, 1024, 32),
                                   (333, 4096, 128), (130, 8192, 64), (70001, 160, 32), (9, 65536, 128)])
def test_int4(elmo, N, L, D, G, zeros):
    (W, s, z), X = _int4(L, D, G, L + N, zeros), _x(N, D, N)
    print(f"  int4 N={N} L={L} D={D} G={G} zeros={zeros}", flush=True)
    y = elmo.w4_matvec(W, X, wfmt=elmo.ELMO_W_INT4, scales=s, zeros=z)
    c, x = _codes(W).double(), X.cpu().double()
    sc = s.cpu().double().repeat_interleave(G, 1)
    zp = z.cpu().double().repeat_interleave(G, 1) if zeros else torch.full_like(c, 8.0)
    _check(y, x @ ((c - zp) * sc).t(), (16 + D / 128) * U * (x.abs() @ ((c + zp) * sc.abs()).t()))


def test_every_code_of_both_formats(elmo):
    """One feature at a time: each product comes back exactly."""
    D = 256
    X = torch.zeros((32, D), dtype=torch.bfloat16, device="cuda")
    ks = torch.arange(32) * 8 + torch.arange(32) % 8
    X[torch.arange(32), ks] = 1.0
    raw = (torch.arange(16)[:, None] * 17).expand(16, D // 2).to(torch.uint8)     # label j: code j everywhere
    for e in (0, 1, 60, 127, 200, 250):
        W = torch.cat([raw, torch.full((16, D // 32), e, dtype=torch.uint8)], 1).contiguous().cuda()
        y = elmo.w4_matvec(W, X).cpu().double()
        want = E2M1 * 2.0 ** (e - 127)
        if e == 0:                                                                # below the normal range: not pinned
            assert y.abs().max() <= 6 * 2.0**-127
        else:
            assert torch.equal(y, want.expand(32, 16))
    s = torch.full((16, D // 32), 0.5, dtype=torch.bfloat16, device="cuda")
    y = elmo.w4_matvec(raw.contiguous().cuda(), X, wfmt=elmo.ELMO_W_INT4, scales=s).cpu()
    assert torch.equal(y, ((torch.arange(16) - 8) * 0.5).expand(32, 16))


def test_feature_order(elmo):
    """Distinct powers of two per feature position within a byte, word and block: sums name their terms."""
    D = 512
    for fmt in (elmo.ELMO_W_MXFP4, elmo.ELMO_W_INT4):
        for k in (0, 1, 2, 3, 7, 8, 31, 32, 63, 64, 127, 128, 255, 256, 511):
            X = torch.zeros((1, D), dtype=torch.bfloat16, device="cuda")
            X[0, k] = 1.0
            g = torch.Generator().manual_seed(k)
            if fmt == elmo.ELMO_W_MXFP4:
                W = _mx(40, D, k)
                assert torch.equal(elmo.w4_matvec(W, X)[0].cpu().double(), _mx_values(W, D)[:, k])
            else:
                W, s, z = _int4(40, D, 32, k, True)
                want = (_codes(W).double()[:, k] - z.cpu().double()[:, k // 32]) * s.cpu().double()[:, k // 32]
                got = elmo.w4_matvec(W, X, wfmt=fmt, scales=s, zeros=z)[0].cpu().double()
                assert (got - want).abs().max() <= 2.0**-22 * 16 * 0.05


@pytest.mark.parametrize("dtype,unit", [(torch.float32, 0.0), (torch.bfloat16, 2.0**-8), (torch.float16, 2.0**-11)])
def test_output_types_and_pitches(elmo, dtype, unit):
    N, L, D = 3, 1001, 768
    W, X = _mx(L, D, 3), _x(N, D, 3, pitch=24)
    wide = torch.zeros((N, L + 11), dtype=dtype, device="cuda")
    y = elmo.w4_matvec(W, X, out=wide[:, 5:5 + L])
    w, x = _mx_values(W, D), X.cpu().double()
    _check(y, x @ w.t(), (D / 32 + 48) * U * (x.abs() @ w.abs().t()), unit)
    assert bool((wide[:, :5] == 0).all()) and bool((wide[:, 5 + L:] == 0).all())
    W, s, z = _int4(L, D, 64, 5, True)
    y = elmo.w4_matvec(W, X, wfmt=elmo.ELMO_W_INT4, scales=s, zeros=z, out_dtype=dtype)
    assert y.dtype == dtype and bool(torch.isfinite(y).all())


def test_nan_stays_in_its_row_and_label(elmo):
    N, L, D = 6, 100, 512
    W, X = _mx(L, D, 9), _x(N, D, 9)
    W[37, D // 2 + 3] = 255
    X[4, 100] = float("nan")
    y = elmo.w4_matvec(W, X).isnan()
    want = torch.zeros((N, L), dtype=torch.bool, device="cuda")
    want[4] = True
    want[:, 37] = True
    assert torch.equal(y, want)
    W, s, z = _int4(L, D, 64, 9, True)
    s[37, 2] = float("nan")
    assert torch.equal(elmo.w4_matvec(W, X, wfmt=elmo.ELMO_W_INT4, scales=s, zeros=z).isnan(), want)


def test_agrees_with_the_framework_logits(elmo):
    """Features that E4M3 holds: elmo_xmc_logits on the same MXFP4 rows computes the same numbers."""
    L, D = 2000, 512
    W, X = _mx(L, D, 1), _x(8, D, 1).float().to(torch.float8_e4m3fn).to(torch.bfloat16)
    a, b = elmo.w4_matvec(W, X), elmo.logits(W, X, 0, L, wfmt=elmo.ELMO_W_MXFP4)
    w, x = _mx_values(W, D), X.cpu().double()
    assert bool(((a - b).abs().cpu().double() <= 2 * (D / 32 + 48) * U * (x.abs() @ w.abs().t())).all())


def test_other_stream_repeats(elmo):
    W, X = _mx(5000, 1024, 2), _x(7, 1024, 2)
    a = elmo.w4_matvec(W, X)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = elmo.w4_matvec(W, X)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_refusals(elmo):
    W, X = _mx(10, 256, 1), _x(2, 256, 1)
    assert elmo.w4_matvec(W, X[:0]).shape == (0, 10)
    with pytest.raises(elmo.ElmoError):
        elmo.w4_matvec(W, _x(33, 256, 1))
    with pytest.raises(elmo.ElmoError):
        elmo.w4_matvec(W, _x(2, 256, 1, pitch=4))                 # rows not 16-byte aligned
    with pytest.raises(elmo.ElmoError):
        elmo.w4_matvec(_mx(10, 128, 1), _x(2, 128, 1))            # D % 256
    with pytest.raises(ValueError):
        elmo.w4_matvec(W, _x(2, 512, 1))
    with pytest.raises(ValueError):
        elmo.w4_matvec(W, X.float())
    with pytest.raises(ValueError):
        elmo.w4_matvec(W, X, scales=torch.ones((10, 8), dtype=torch.bfloat16, device="cuda"))
    I, s, z = _int4(10, 256, 32, 1, True)
    with pytest.raises(ValueError):
        elmo.w4_matvec(I, X, wfmt=elmo.ELMO_W_INT4)
    with pytest.raises(ValueError):
        elmo.w4_matvec(I, X, wfmt=elmo.ELMO_W_INT4, scales=s.float())
    with pytest.raises(ValueError):
        elmo.w4_matvec(I, X, wfmt=elmo.ELMO_W_INT4, scales=s, zeros=z[:, :4])
    with pytest.raises(elmo.ElmoError):
        elmo.w4_matvec(I, X, wfmt=elmo.ELMO_W_INT4, scales=s[:, :1].contiguous())   # groups of 256
    with pytest.raises(TypeError):
        elmo.w4_matvec(W, X, wfmt=elmo.ELMO_W_E4M3)
    with pytest.raises(TypeError):
        elmo.w4_matvec(W, X, out_dtype=torch.float64)


@pytest.mark.parametrize("fmt,N,L,D,G", [("mx", 29, 17000, 3840, 32), ("mx", 32, 16500, 4096, 32), ("mx", 16, 16401, 6144, 32),
                                         ("mx", 18, 20000, 2560, 32), ("int4", 21, 16500, 7296, 128), ("int4", 24, 17003, 4832, 32),
                                         ("int4", 9, 16400, 8192, 64), ("int4", 32, 20001, 2080, 32)])
def test_feature_rows_beyond_lds(elmo, fmt, N, L, D, G):
    """Many labels and more features than fit LDS at once (FP32 results summed over panels of D,
    16-bit ones in one go), and just as many as fit; float64 products on the GPU in slices."""
    print(f"  {fmt} N={N} L={L} D={D} G={G}", flush=True)
    X = _x(N, D, N)
    x = X.double()
    if fmt == "mx":
        W, kw, eps = _mx(L, D, L), {}, (D / 32 + 56) * U
    else:
        W, s, z = _int4(L, D, G, L, True)
        kw, eps = dict(wfmt=elmo.ELMO_W_INT4, scales=s, zeros=z), (24 + D / 128) * U      # (panels: a few sums more)
    y, h = elmo.w4_matvec(W, X, **kw), elmo.w4_matvec(W, X, out_dtype=torch.bfloat16, **kw)
    table = E2M1.cuda()
    for a in range(0, L, 4096):
        r = W[a:a + 4096]
        c = torch.stack([r[:, :D // 2] & 15, r[:, :D // 2] >> 4], 2).flatten(1).int()
        if fmt == "mx":
            w = table[c] * torch.exp2(r[:, D // 2:].double() - 127).repeat_interleave(32, 1)
            size = w.abs()
        else:
            sc, zp = (t[a:a + 4096].double().repeat_interleave(G, 1) for t in (s, z))
            w, size = (c.double() - zp) * sc, (c.double() + zp) * sc.abs()
        ref, tol = x @ w.t().contiguous(), eps * (x.abs() @ size.t().contiguous())
        off = (y[:, a:a + 4096].double() - ref).abs()
        assert bool((off <= tol).all()), f"off by {off.max():.3e}, {(off / tol).max():.3g} of the tolerance"
        off = (h[:, a:a + 4096].double() - ref).abs()
        assert bool((off <= tol + 2.0**-8 * ref.abs()).all())


def test_integer_codes_of_more_labels_than_one_launch_holds(elmo):
    """2^27 + 21 labels of 1920 features with 32 rows and 16-bit results: a block per 16 labels would be
    more than 2^32 threads, and offsets pass 2^36 bytes. Stretches equal their own calls bit for bit."""
    L, N, D, G = (1 << 27) + 21, 32, 1920, 128
    need = L * (D // 2 + 2 * (D // G) + 2 * N) + (4 << 30)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of free device memory")
    X = _x(N, D, 5)
    W = torch.empty((L, D // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((L, D // G), dtype=torch.bfloat16, device="cuda")
    stretches = [(0, 37), ((1 << 26) - 16, (1 << 26) + 16), ((1 << 27) - 16, L)]
    for a, b in stretches:
        W[a:b], s[a:b], _ = _int4(b - a, D, G, a % 1000, False)
    y = elmo.w4_matvec(W, X, wfmt=elmo.ELMO_W_INT4, scales=s, out_dtype=torch.bfloat16)
    for a, b in stretches:
        assert torch.equal(y[:, a:b], elmo.w4_matvec(W[a:b], X, wfmt=elmo.ELMO_W_INT4, scales=s[a:b], out_dtype=torch.bfloat16))
    a, b = stretches[-1]
    c, x, sc = _codes(W[a:b]).double(), X.cpu().double(), s[a:b].cpu().double().repeat_interleave(G, 1)
    ref = x @ ((c - 8) * sc).t()
    _check(y[:, a:b], ref, (12 + D / 128) * U * (x.abs() @ ((c + 8) * sc.abs()).t()), 2.0**-8)
    del W, s, y
    torch.cuda.empty_cache()
