"""Calls of more rows, or labels, than one launch has threads for (2^32): the same ones again and again, whose results are
all the same."""
import pytest
import torch

from test_gpu_linear_logprobs import BF, HALF, LEAST, _case, _gradients, _near, elmo  # noqa: F401

pytestmark = pytest.mark.gpu


def _repeated(base, times, more):
    """`base` one below the other, and its first `more` rows."""
    n = base.shape[0]
    t = torch.empty((n * times + more, *base.shape[1:]), dtype=base.dtype, device=base.device)
    t[:n * times].view(times, n, *base.shape[1:]).copy_(base.expand(times, *base.shape))
    t[n * times:] = base[:more]
    return t


def _same(got, base, times, more):
    n = base.shape[0]
    head = got[:n * times].view(times, n, *base.shape[1:])
    return all(bool((head[i:i + 64] == base).all()) for i in range(0, times, 64)) and bool((got[n * times:] == base[:more]).all())


@pytest.mark.parametrize("D,times", [(64, 1 << 14), (2112, 1 << 12)])
def test_quantise_many_rows(elmo, D, times):  # noqa: F811
    """Over 2^26 rows of a wave each, over 2^24 rows of a block each."""
    torch.cuda.empty_cache()
    g = torch.Generator(device="cuda").manual_seed(2)
    base = torch.randn((4096, D), generator=g, device="cuda").to(BF)
    codes, scales = elmo.i8_quantize(base)
    x = _repeated(base, times, 70)
    print(f"  i8_quantize {tuple(x.shape)}", flush=True)
    c, s = elmo.i8_quantize(x)
    assert _same(c, codes, times, 70) and _same(s, scales, times, 70)
    del x, c, s
    torch.cuda.empty_cache()


def test_log_probabilities_of_many_rows(elmo):  # noqa: F811
    """Over 2^26 rows, which are the same 4,096 again and again: all their results and gradients are the same, and near
    float64's."""
    torch.cuda.empty_cache()
    X, W, ids, up, _ = _case(4096, 64, 32, 1, BF, seed=9)
    times = 1 << 14
    many, many_ids, many_up = (_repeated(t, times, 70) for t in (X, ids, up))
    print(f"  linear_logprobs {tuple(many.shape)}", flush=True)
    r = elmo.linear_logprobs(many, W, many_ids)
    z = X.double() @ W.double().t()
    lse = torch.logsumexp(z, 1)
    want = z.gather(1, ids.long()) - lse[:, None]
    assert float((r.logp[:4096].double() - want).abs().max()) < 1e-5
    assert float((r.row_max[:4096].double() + r.log_sum[:4096].double() - lse).abs().max()) < 1e-5
    for t in r:
        assert _same(t, t[:4096].clone(), times, 70)
    dx, _ = elmo.linear_logprobs_backward(many, W, many_ids, r, many_up, need_dw=False)
    dX, _, tX, _ = _gradients(X, W, ids, up, None)
    _near(dx[:4096], dX, tX + HALF[BF] * (dX.abs() + tX) + LEAST[BF], "dX")
    assert _same(dx, dx[:4096].clone(), times, 70)
    del many, r, dx
    torch.cuda.empty_cache()


def test_8_bit_products_of_many_labels(elmo):  # noqa: F811
    """2^31 - 1 labels of 64 features, 2^20 of them again and again."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 180 << 30:
        pytest.skip("needs 180 GiB of device memory")
    g = torch.Generator(device="cuda").manual_seed(3)
    base = torch.randint(-127, 128, (1 << 20, 64), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(1 << 20, generator=g, device="cuda")
    x, sx = torch.randint(-127, 128, (1, 64), generator=g, device="cuda", dtype=torch.int8), torch.ones(1, device="cuda")
    want = elmo.i8_matmul(x, sx, base, sw)[0]
    W, s = _repeated(base, 2047, (1 << 20) - 1), _repeated(sw, 2047, (1 << 20) - 1)
    print(f"  i8_matmul {tuple(x.shape)} {tuple(W.shape)}", flush=True)
    y = elmo.i8_matmul(x, sx, W, s)[0]
    assert _same(y, want, 2047, (1 << 20) - 1)
    del W, s, y
    torch.cuda.empty_cache()
