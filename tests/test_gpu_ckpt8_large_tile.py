"""The weight gradient from 8-bit checkpoints in its 256 x 256 tile, which wide layers take, against
float64 on the GPU. (test_lm_launches.py holds that these shapes take it, one segment of tokens and
several.)

Tolerance (u = 2^-24): the products are exact; matrix products of 16 tokens round at most 16 times
relative to their own terms, the chain of T / 16 of them once each relative to the sum of
magnitudes so far, and at most 16 partial sums are added: (T / 16 + 32) u sum|dy x|."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
# (T, O, D): no whole tiles in O and D, no whole stages in T; even and odd numbers of stages
SHAPES = [(1001, 2056, 4128), (2049, 2056, 4128), (2023, 4088, 4064), (4001, 2056, 2080), (8005, 1800, 1824),
          (16001, 1000, 2016), (16384, 2048, 4096)]


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def _saved(T, D, seed):
    """(codes, scales, values float64) on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8, device="cuda")

    codes, scales = draw(0, 127, (T, D)) + 128 * draw(0, 2, (T, D)), draw(115, 123, (T, D // 32))
    return codes, scales, codes.view(torch.float8_e4m3fn).double() * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _within(got, ref, tol):
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), f"off by {off.max():.3e}, {(off / tol.clamp(min=1e-300)).max():.3g} of the tolerance"


@pytest.mark.parametrize("T,O,D", SHAPES)
def test_against_float64(elmo, T, O, D):
    codes, scales, x = _saved(T, D, T)
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    pitched = torch.full((T, O + 24), float("nan"), dtype=torch.bfloat16, device="cuda")   # beside the rows
    pitched[:, :O] = torch.randn((T, O), generator=g, device="cuda")
    dy = pitched[:, :O].contiguous()
    print(f"  wgrad T={T} O={O} D={D}", flush=True)
    t = dy.double().t().contiguous()
    ref, tol = t @ x, (T / 16 + 32) * U * (t.abs() @ x.abs())
    a = elmo.ckpt8_weight_grad(pitched[:, :O], codes, scales)
    _within(a, ref, tol)
    assert torch.equal(a, elmo.ckpt8_weight_grad(dy, codes, scales))                        # and it repeats
    base = torch.randn((O, D), generator=g, device="cuda") * a.abs().mean()
    c = elmo.ckpt8_weight_grad(dy, codes, scales, out=base.clone(), accumulate=True)
    _within(c.double() - base.double(), ref, tol + 4 * U * (base.double().abs() + ref.abs()))


@pytest.mark.parametrize("T,O,D", [(1001, 2056, 4128), (1801, 1800, 1824)])
def test_one_hot_tokens(elmo, T, O, D):
    """A single 1 per token (and per output) picks rows of x exactly: every index of both operands is named."""
    rows = 8005 if O == 1800 else T                                # (the second shape: zeros, then the tokens)
    codes, scales, x = _saved(rows, D, 4)
    g = torch.Generator(device="cuda").manual_seed(3)
    n = min(T, O)
    tokens = rows - n + torch.randperm(n, generator=g, device="cuda")
    at = torch.randperm(O, generator=g, device="cuda")[:n]
    dy = torch.zeros((rows, O), dtype=torch.bfloat16, device="cuda")
    dy[tokens, at] = 1.0
    want = torch.zeros((O, D), dtype=torch.float64, device="cuda")
    want[at] = x[tokens]
    assert torch.equal(elmo.ckpt8_weight_grad(dy, codes, scales).double(), want)


@pytest.mark.parametrize("T,O,D", [(1001, 2056, 4128), (4001, 2056, 2080)])
def test_nan_reaches_its_outputs_only(elmo, T, O, D):
    codes, scales, _ = _saved(T, D, 1)
    dy = torch.ones((T, O), dtype=torch.bfloat16, device="cuda")
    codes[T - 1, 3], codes[500, D - 40], scales[9, 1] = 0x7F, 0xFF, 255
    dy[700, O - 1] = float("nan")
    want = torch.zeros((O, D), dtype=torch.bool, device="cuda")
    want[:, 3], want[:, D - 40], want[:, 32:64], want[O - 1] = True, True, True, True
    assert torch.equal(elmo.ckpt8_weight_grad(dy, codes, scales).isnan(), want)


def test_graph_replays(elmo):
    """The product and the join captured once, replayed with new gradients and eager work in between."""
    T, O, D = 4001, 2056, 2080
    codes, scales, _ = _saved(T, D, 2)
    dy = torch.randn((T, O), device="cuda").to(torch.bfloat16)
    ws = torch.empty(elmo.lib().elmo_ckpt8_weight_grad_workspace_bytes(T, O, D), dtype=torch.uint8, device="cuda")
    out = torch.zeros((O, D), device="cuda")
    elmo.ckpt8_weight_grad(dy, codes, scales, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        elmo.ckpt8_weight_grad(dy, codes, scales, out=out, workspace=ws)
    for _ in range(4):
        dy.copy_(torch.randn((T, O), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, elmo.ckpt8_weight_grad(dy, codes, scales))
