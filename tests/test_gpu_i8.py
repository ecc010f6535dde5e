"""Products in 8-bit integers against plain integer and float64 arithmetic on the CPU. Codes are compared for
equality (the quotient's rounding is defined exactly); results carry the roundings of the sum to binary32, of the two
scales' products and of the result: 3 u + half a unit of its type, relative."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def _plain_codes(x):
    x = x.cpu().double()
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(x * 127.0 / torch.where(top > 0, top, torch.ones_like(top)))
    return q.to(torch.int8), (top[:, 0] / 127.0).float()


def _check_codes(elmo, x):
    codes, scales = elmo.i8_quantize(x)
    want, s = _plain_codes(x)
    assert torch.equal(codes.cpu(), want), f"{int((codes.cpu() != want).sum())} codes differ"
    assert torch.equal(scales.cpu(), s)


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("N,D", [(1, 64), (3, 128), (5, 2048), (7, 2112), (2, 8192), (3, 8256), (1, 65536), (1000, 768)])
def test_codes(elmo, N, D, dtype):
    g = torch.Generator().manual_seed(N + D)
    x = (torch.randn((N, D), generator=g) * torch.exp(torch.randn((D,), generator=g))).to(dtype).cuda()
    print(f"  i8_quantize {N} x {D} {dtype}", flush=True)
    _check_codes(elmo, x)


def test_codes_at_ties(elmo):
    """Halves go to the even code, their neighbours to the nearest, at rows of any size."""
    for top in (127.0, 254.0, 1.0, 3.0, 1.5e-38, 2.0**-140, 3.0e38, 16777213.0):
        k = torch.arange(-127, 128, dtype=torch.float64)
        tie = (k + 0.5).clamp(-127, 127) * top / 127.0
        v = torch.cat([tie, torch.tensor([top], dtype=torch.float64)]).float()
        rows = torch.stack([v, torch.nextafter(v, torch.full_like(v, -float("inf"))), torch.nextafter(v, torch.full_like(v, float("inf")))])
        rows[:, -1] = float(torch.tensor(top, dtype=torch.float32))
        rows = rows.clamp(-rows[0, -1], rows[0, -1])
        _check_codes(elmo, rows.cuda())


def test_codes_of_odd_rows(elmo):
    x = torch.randn((5, 256), device="cuda")
    x[1] = 0.0
    x[2, 200] = float("nan")
    x[3, 7] = float("-inf")
    codes, scales = elmo.i8_quantize(x)
    assert bool((codes[1:4] == 0).all()) and scales[1] == 0 and bool(scales[2:4].isnan().all())
    _check_codes(elmo, x[::4])
    wide = torch.randn((6, 336), device="cuda", dtype=BF)
    _check_codes(elmo, wide[:, :320])
    _check_codes(elmo, wide[::2, 16:336])


def _check_product(elmo, N, L, D, out, pad=0, shift=0, seed=0, full=False):
    g = torch.Generator().manual_seed(seed + N + L + D)
    lo = -128 if full else -127
    X = torch.randint(lo, 128, (N, D), generator=g, dtype=torch.int8)
    W = torch.randint(lo, 128, (L, D), generator=g, dtype=torch.int8)
    if full:
        X[0], W[0] = -128, -128
        X[-1], W[-1] = 127, -128
    sx, sw = torch.rand((N,), generator=g) + 0.01, torch.rand((L,), generator=g) * 1e-3
    buf = torch.full((N * (L + pad) + shift,), 7.0, device="cuda", dtype=out)
    y = buf[shift:].view(N, L + pad)[:, :L]
    print(f"  i8_matmul {N} x {L} x {D} {out} pitch {L + pad} + {shift}", flush=True)
    elmo.i8_matmul(X.cuda(), sx.cuda(), W.cuda(), sw.cuda(), out=y)
    want = (X.double() @ W.double().t()) * sx.double()[:, None] * sw.double()
    tol = want.abs() * (3 * U + HALF[out] * (1 + 4 * U)) + (2.0**-25 if out == HF else 0.0)
    off = (y.cpu().double() - want).abs()
    assert bool((off <= tol).all()), f"off by {(off / want.abs()).nan_to_num().max():.3e} relative"
    rest = buf.clone()
    rest[shift:].view(N, L + pad)[:, :L] = 7.0
    assert bool((rest == 7.0).all()), "written beside the results"


@pytest.mark.parametrize("out", [F32, BF, HF])
@pytest.mark.parametrize("N,L,D", [(1, 1, 64), (1, 17, 128), (2, 4099, 192), (16, 515, 704), (17, 1000, 768), (31, 33, 4096), (32, 70003, 64),
                                   (33, 5, 64), (64, 257, 128), (100, 1030, 1088), (256, 256, 64), (257, 513, 320), (300, 7000, 256)])
def test_products(elmo, N, L, D, out):
    _check_product(elmo, N, L, D, out)


@pytest.mark.parametrize("N,L,D", [(1, 4096, 16384), (16, 128, 65536), (40, 300, 65536), (700, 260, 8192), (2000, 2048, 512)])
def test_long(elmo, N, L, D):
    """The largest whole sums, runs of K that are summed apart, many tiles."""
    _check_product(elmo, N, L, D, F32, full=True)
    _check_product(elmo, N, L, D, BF)


@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 1), (8, 8), (5, 3)])
@pytest.mark.parametrize("N", [3, 20, 90])
def test_result_pitches(elmo, N, pad, shift):
    for out in (F32, BF, HF):
        for L in (301, 512):
            _check_product(elmo, N, L, 128, out, pad, shift)


def test_scales_out_of_range_stay(elmo):
    X = torch.ones((40, 64), device="cuda", dtype=torch.int8)
    W = torch.ones((50, 64), device="cuda", dtype=torch.int8)
    sx, sw = torch.ones(40, device="cuda"), torch.ones(50, device="cuda")
    sx[3], sw[7] = float("nan"), float("inf")
    for n in (8, 40):
        y = elmo.i8_matmul(X[:n], sx[:n], W, sw, out_dtype=F32)
        bad = y.isnan()
        assert bool(bad[3].all()) and int(bad.sum()) == 50
        good = torch.arange(n, device="cuda") != 3
        assert bool((y[good, 7] == float("inf")).all()) and bool((y[good][:, :7] == 64).all())


def test_no_rows_graph_and_workspace(elmo):
    W = torch.randint(-127, 128, (300, 4096), device="cuda", dtype=torch.int8)
    sw = torch.rand(300, device="cuda")
    assert elmo.i8_matmul(W[:0], sw[:0], W, sw).shape == (0, 300)
    assert elmo.i8_quantize(torch.empty((0, 64), device="cuda"))[0].shape == (0, 64)
    for n in (5, 60):
        x = torch.randn((n, 4096), device="cuda", dtype=BF)

        def call(ws=None):
            return elmo.i8_matmul(*elmo.i8_quantize(x), W, sw, workspace=ws)
        want = call()
        need = elmo.lib().elmo_i8_matmul_workspace_bytes(n, 300, 4096)
        assert torch.equal(call(torch.full((need + 16,), 255, device="cuda", dtype=torch.uint8)), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for _ in range(3):
            x.normal_()
            want = call()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_refusals(elmo):
    X, W = (torch.ones((4, 128), device="cuda", dtype=torch.int8) for _ in range(2))
    s = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        elmo.i8_matmul(X.float(), s, W, s)
    with pytest.raises(ValueError):
        elmo.i8_matmul(X[:, :64], s, W[:, :64], s)
    with pytest.raises(ValueError):
        elmo.i8_matmul(X, s, W[:, :64].contiguous(), s)
    with pytest.raises(ValueError):
        elmo.i8_matmul(X, s.double(), W, s)
    with pytest.raises(ValueError):
        elmo.i8_matmul(X, s, W, s, out=torch.empty((4, 5), device="cuda"))
    with pytest.raises(TypeError):
        elmo.i8_matmul(X, s, W, s, out_dtype=torch.int32)
    with pytest.raises(elmo.ElmoError):
        elmo.i8_matmul(X[:, :96].contiguous(), s, W[:, :96].contiguous(), s)
    with pytest.raises(elmo.ElmoError):
        elmo.i8_quantize(torch.ones((4, 96), device="cuda"))
    with pytest.raises(TypeError):
        elmo.i8_quantize(torch.ones((4, 64), device="cuda", dtype=torch.float64))
    with pytest.raises(elmo.ElmoError):
        elmo.i8_quantize(torch.ones((4, 65), device="cuda")[:, :64])
