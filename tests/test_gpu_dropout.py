"""Dropout from the counter-based generator: its draws against a plain Philox4x32-10 in numpy, its results bit
for bit against binary32 arithmetic rounded once."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def draws(first, n, seed, step):
    """The 16 random bits of elements first .. first + n - 1."""
    b = np.arange(first >> 3, (first + n + 7) >> 3, dtype=np.uint64)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [b & low, b >> half, np.full_like(b, step & 0xFFFFFFFF), np.full_like(b, step >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> half) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> half) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    w = np.stack(c, 1).astype("<u4").view("<u2").reshape(-1)
    return torch.from_numpy(w[first & 7:(first & 7) + n].astype(np.int32))


def plain(x, p, seed, step, residual=None, first=0):
    limit = int(p * 65536 + 0.5)
    keep = (draws(first, x.numel(), seed, step) >= limit).view(x.shape)
    f = np.float32(65536) / np.float32(65536 - limit) if limit < 65536 else np.float32(0)
    y = torch.where(keep, x.cpu().float() * float(f), torch.zeros(()))
    if residual is not None:
        y = residual.cpu().float() + y
    return y.to(x.dtype)


def _same(a, b):
    return torch.equal(a.cpu().view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.cpu().view(torch.int16 if b.element_size() == 2 else torch.int32))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 7), (1, 8), (2, 3), (3, 64), (5, 77), (64, 768), (33, 1000), (1000, 515)])
def test_sizes(elmo, T, D, dtype, residual):
    x, r = torch.randn((T, D), device="cuda").to(dtype), torch.randn((T, D), device="cuda").to(dtype)
    r = r if residual else None
    for p, seed, step in ((0.1, 3, 0), (0.5, 0xFEDCBA9876543210, 0x123456789AB)):
        print(f"  dropout {T} x {D} {dtype} p={p}", flush=True)
        assert _same(elmo.dropout(x, p, seed, step, residual=r), plain(x, p, seed, step, r))
    assert _same(elmo.dropout_backward(x, p, seed, step), plain(x, p, seed, step))


@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0**-16, 0.999999, 1.0])
def test_probabilities(elmo, p):
    x = torch.randn((40, 1024), device="cuda")
    y = elmo.dropout(x, p, 9)
    assert _same(y, plain(x, p, 9, 0))
    if p in (0.0, 1e-6):
        assert torch.equal(y, x)
    if p == 1.0:
        assert bool((y == 0).all())
        assert torch.equal(elmo.dropout(x, 1.0, 9, residual=x), x)


def test_pitches_alignment_and_in_place(elmo):
    for dtype in (F32, BF, HF):
        for D, pad, shift in ((64, 8, 0), (64, 3, 0), (63, 1, 1), (128, 0, 3), (8, 8, 8)):
            buf = [torch.randn(20 * (D + pad) + shift, device="cuda").to(dtype) for _ in range(3)]
            x, r, out = (b[shift:].view(20, D + pad)[:, :D] for b in buf)
            keep = buf[2].clone()
            want = plain(x, 0.3, 5, 6, r)
            assert _same(elmo.dropout(x, 0.3, 5, 6, residual=r, out=out).contiguous(), want)
            keep[shift:].view(20, D + pad)[:, :D] = out
            assert torch.equal(keep, buf[2]), "written beside the results"
            assert _same(elmo.dropout(x, 0.3, 5, 6, residual=r, out=r).contiguous(), want)
            want = plain(x, 0.3, 5, 6)
            assert _same(elmo.dropout(x, 0.3, 5, 6, out=x).contiguous(), want)


def test_parts_draw_what_the_whole_does(elmo):
    x = torch.randn((50, 77), device="cuda")
    y = elmo.dropout(x, 0.4, 11, 2)
    for a, b in ((0, 8), (8, 9), (9, 50)):
        assert torch.equal(elmo.dropout(x[a:b], 0.4, 11, 2, first=a * 77), y[a:b])
    far = (1 << 40) + 5                      # indices past 32 bits
    assert _same(elmo.dropout(x, 0.4, 11, 2, first=far), plain(x, 0.4, 11, 2, first=far))
    assert torch.equal(elmo.dropout(x.view(-1), 0.4, 11, 2).view(50, 77), y)


def test_dropped_values_do_not_matter(elmo):
    x = torch.randn((32, 256), device="cuda")
    y = elmo.dropout(x, 0.5, 1)
    bad = torch.where(draws(0, x.numel(), 1, 0).view(32, 256).cuda() < 32768, float("nan"), x)
    assert torch.equal(elmo.dropout(bad, 0.5, 1), y)


def test_keeps_the_mean(elmo):
    """Over n = 2^22 elements the share kept is within 6 standard deviations of 1 - p, and differs by key."""
    x = torch.ones((1 << 10, 1 << 12), device="cuda")
    a, b, c = (elmo.dropout(x, 0.25, s, t) for s, t in ((1, 0), (2, 0), (1, 1)))
    for y in (a, b, c):
        assert abs(float((y != 0).double().mean()) - 0.75) < 6 * (0.75 * 0.25 / x.numel())**0.5
    for y, z in ((a, b), (a, c), (b, c)):
        both = float(((y != 0) & (z != 0)).double().mean())
        assert abs(both - 0.5625) < 6 * (0.5625 * 0.4375 / x.numel())**0.5


def test_step_on_the_device(elmo):
    """A recorded graph that counts the step up draws what eager calls with whole numbers do."""
    x, r = torch.randn((64, 96), device="cuda", dtype=BF), torch.randn((64, 96), device="cuda", dtype=BF)
    step = torch.zeros(1, device="cuda", dtype=torch.int64)
    assert torch.equal(elmo.dropout(x, 0.2, 4, step), elmo.dropout(x, 0.2, 4, 0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        y = elmo.dropout(x, 0.2, 4, step, residual=r)
        d = elmo.dropout_backward(x, 0.2, 4, step)
    step.zero_()
    for i in range(1, 5):
        want = elmo.dropout(x, 0.2, 4, i, residual=r), elmo.dropout(x, 0.2, 4, i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(d, want[1])


def test_empty_and_refusals(elmo):
    assert elmo.dropout(torch.empty((0, 5), device="cuda"), 0.5, 1).shape == (0, 5)
    assert elmo.dropout(torch.empty((5, 0), device="cuda"), 0.5, 1).shape == (5, 0)
    x = torch.ones((4, 8), device="cuda")
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(elmo.ElmoError):
            elmo.dropout(x, p, 1)
    with pytest.raises(TypeError):
        elmo.dropout(x.double(), 0.5, 1)
    with pytest.raises(ValueError):
        elmo.dropout(x, 0.5, 1, residual=x[:2])
    with pytest.raises(ValueError):
        elmo.dropout(x, 0.5, 1, out=x.to(BF))
    with pytest.raises(ValueError):
        elmo.dropout(x, 0.5, 1, step=torch.zeros(2, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        elmo.dropout(x.t(), 0.5, 1)
    with pytest.raises(ValueError):
        elmo.dropout(x.cpu(), 0.5, 1)
