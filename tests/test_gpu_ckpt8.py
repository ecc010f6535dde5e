"""Activation checkpoints in 8 bits and their use in the backward pass.

Codes and scales are compared bit for bit with a plain float64 form. Tolerances of the rest
(u = 2^-24): the exponential's argument carries 3 roundings of relative size u, so sigmoid is off by
r = (3 |x| + 8) u relative and silu by r + 2 u; Phi by 1.5 (x^2 + 16) u relative (the roundings of
x^2 in the exponent, 9 of the polynomial, the fit's 2e-8); products add one u each; results are
rounded once to their type. Weight gradients: T exact products summed in some order, T u of the sum
of their magnitudes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
UNIT = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0**-24}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
ACTS = ["relu", "silu", "gelu"]


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def _keep(x):
    """(codes, scales, values float64) of the definition, on the CPU."""
    T, D = x.shape
    b = x.cpu().double().view(T, D // 32, 32)
    fin = torch.isfinite(b)
    top = torch.where(fin, b.abs(), torch.zeros_like(b)).amax(2)
    X = torch.full_like(top, -127.0)
    for e in range(-127, 121):                                    # the smallest power that holds the largest
        X = torch.where(top > 448 * 2.0**e, torch.full_like(X, e + 1.0), X)
    q = torch.where(fin, b * torch.exp2(-X)[:, :, None], torch.full_like(b, math.nan))
    a = q.abs()
    unit = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0**-6))) - 3)
    v = torch.round(a / unit) * unit                              # to nearest even (torch.round)
    codes = (v.float() * torch.sign(q).float()).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where((v == 0) & torch.signbit(b), torch.full_like(codes, 128), codes)
    val = torch.copysign(v, b) * torch.exp2(X)[:, :, None]
    return codes.view(T, D), (X + 127).to(torch.uint8), torch.where(fin, val, torch.full_like(val, math.nan)).view(T, D)


def _same_codes(got, ref):
    nan = (ref & 127) == 127
    assert torch.equal((got & 127) == 127, nan)
    assert torch.equal(got[~nan], ref[~nan])


def _x(T, D, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, D + pad), generator=g) * torch.exp2(torch.randint(-6, 7, (1, D + pad), generator=g).float())
    return x.to(dtype).cuda()[:, :D]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D,pad", [(1, 32, 0), (3, 64, 8), (77, 96, 0), (1, 4096, 0), (513, 800, 32), (5000, 32, 0)])
def test_codes_and_restored_values(elmo, T, D, pad, dtype):
    x = _x(T, D, dtype, T + D, pad)
    codes, scales, y = elmo.ckpt8_save(x)
    rc, rs, val = _keep(x)
    assert y is None
    assert torch.equal(scales.cpu(), rs)
    _same_codes(codes.cpu(), rc)
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(elmo.ckpt8_load(codes, scales, dtype=out).cpu().double(), val)
    h = elmo.ckpt8_load(codes, scales, dtype=torch.float16)
    assert torch.equal(h.cpu(), val.float().to(torch.float16))


def test_block_scale_edges(elmo):
    """Largest elements around 448 2^X, powers of two, subnormals, the type's extremes, zeros and ties."""
    tops = [0.0, 1.0, 1.75, 1.7500001, 1.75 * 2**-20, 2.0**-126, 2.0**-127, 2.0**-149, 2.0**-135, 448.0, 448.00003,
            447.99997, 3.4028234e38, 2.0**127, 1.75 * 2.0**127, 2.0**-119, 2.0**-118, 1.75 * 2.0**-119]
    g = torch.Generator().manual_seed(2)
    rows = []
    for t in tops:
        r = (torch.rand(32, generator=g) * 2 - 1) * t
        r[5] = -t
        r[6:10] = torch.tensor([t / 16, t / 32, 17 / 16 * t / 32, -0.0])
        rows.append(r)
    # every tie between two neighbouring codes at scale 1 (a largest element of 448 fixes it)
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (grid[:-1] + grid[1:]) / 2
    for i in range(0, mid.numel(), 31):
        r = torch.zeros(32)
        r[0] = 448.0
        m = mid[i:i + 31]
        r[1:1 + m.numel()] = m
        rows += [r, -r]
    x = torch.stack(rows).cuda()
    codes, scales, _ = elmo.ckpt8_save(x)
    rc, rs, val = _keep(x)
    assert torch.equal(scales.cpu(), rs)
    _same_codes(codes.cpu(), rc)
    # FP32's largest values round up to 256 2^120 = 2^128, which FP32 holds as infinity
    assert torch.equal(elmo.ckpt8_load(codes, scales, dtype=torch.float32).cpu(), val.float())


def test_every_bf16_value(elmo):
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)[torch.randperm(65536, generator=torch.Generator().manual_seed(1))].view(-1, 64).cuda()
    codes, scales, _ = elmo.ckpt8_save(x)
    rc, rs, _ = _keep(x)
    assert torch.equal(scales.cpu(), rs)
    _same_codes(codes.cpu(), rc)


def test_nan_and_infinity_keep_to_themselves(elmo):
    x = _x(4, 64, torch.float32, 3)
    clean = elmo.ckpt8_save(x.clone())
    x[1, 7], x[1, 40], x[2, 63] = math.nan, math.inf, -math.inf
    codes, scales, y = elmo.ckpt8_save(x, act="relu")
    bad = ~torch.isfinite(x)
    assert bool(((codes[bad] & 127) == 127).all())
    same = ~(bad.view(4, 2, 32).any(2, keepdim=True).expand(4, 2, 32).reshape(4, 64))
    assert torch.equal(codes[same], clean[0][same])
    rc, rs, _ = _keep(x)
    assert torch.equal(scales.cpu(), rs)
    _same_codes(codes.cpu(), rc)
    assert y[1, 7].isnan() and y[1, 40] == math.inf and y[2, 63] == 0
    dx = elmo.ckpt8_act_grad(torch.ones_like(x), codes, scales, "silu")
    assert torch.equal(dx.isnan(), bad)


def _act64(x, act):
    if act == "relu":
        return torch.relu(x), (x > 0).double(), torch.zeros_like(x), torch.zeros_like(x)
    if act == "silu":
        s = torch.sigmoid(x)
        r = (3 * x.abs() + 8) * U
        q = 1 - s
        return x * s, s * (1 + x * q), (r + 2 * U) * (x * s).abs(), s * (r * (1 + x.abs() * q) + x.abs() * (s * r + U) + 3 * U)
    c = 0.5 * torch.erfc(-x / math.sqrt(2))
    f = torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    r = 1.5 * (x * x + 16) * U
    return x * c, c + x * f, (r + U) * (x * c).abs(), r * (c + x.abs() * f) + 2 * U


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_activation_and_its_gradient(elmo, act, dtype):
    for T, D, pad in ((1, 32, 0), (37, 96, 8), (300, 1024, 0)):
        x = _x(T, D, dtype, D, pad)
        x[0, 0] = 0.0
        dy = _x(T, D, dtype, D + 1, pad)
        codes, scales, y = elmo.ckpt8_save(x, act=act)
        assert torch.equal(codes, elmo.ckpt8_save(x)[0])
        val, _, tol, _ = _act64(x.cpu().double(), act)
        off = (y.cpu().double() - val).abs()
        assert bool((off <= tol + UNIT[dtype] * val.abs() + TINY[dtype]).all()), off.max()
        kept = _keep(x)[2]
        _, slope, _, tol = _act64(kept, act)
        d = dy.cpu().double()
        want = d * slope
        got = elmo.ckpt8_act_grad(dy, codes, scales, act)
        off = (got.cpu().double() - want).abs()
        assert bool((off <= tol * d.abs() + (UNIT[dtype] + U) * want.abs() + TINY[dtype]).all()), off.max()
        place = dy.clone() if pad == 0 else dy
        over = elmo.ckpt8_act_grad(place, codes, scales, act, out=place)
        assert over.data_ptr() == place.data_ptr() and torch.equal(over, got)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_gradient_against_differences(elmo, act):
    """act' of the saved values against central differences of the float64 activation."""
    x = torch.linspace(-6, 6, 1024).view(8, 128).cuda()
    codes, scales, _ = elmo.ckpt8_save(x, act=act)
    kept = elmo.ckpt8_load(codes, scales, dtype=torch.float32).cpu().double()
    h = 1e-4
    ref = (_act64(kept + h, act)[0] - _act64(kept - h, act)[0]) / (2 * h)
    got = elmo.ckpt8_act_grad(torch.ones_like(x), codes, scales, act).cpu().double()
    assert (got - ref).abs().max() < 2e-6                         # h^2 times the third derivative, and binary32


def _saved(T, D, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 127, (T, D), generator=g, dtype=torch.uint8) + 128 * torch.randint(0, 2, (T, D), generator=g, dtype=torch.uint8)
    scales = torch.randint(115, 123, (T, D // 32), generator=g, dtype=torch.uint8)
    val = codes.view(torch.float8_e4m3fn).double() * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return codes.cuda(), scales.cuda(), val


@pytest.mark.parametrize("T,O,D", [(1, 8, 32), (5, 64, 64), (31, 128, 128), (33, 136, 160), (64, 768, 768), (1001, 200, 96),
                                   (4097, 264, 288), (513, 8, 1056), (700, 1000, 32), (20000, 128, 256), (3000, 520, 544)])
def test_weight_gradient(elmo, T, O, D):
    codes, scales, x = _saved(T, D, T)
    g = torch.Generator().manual_seed(T + 1)
    dy = torch.randn((T, O + 16), generator=g).to(torch.bfloat16)[:, :O]
    print(f"  wgrad T={T} O={O} D={D}", flush=True)
    pitched = torch.zeros((T, O + 16), dtype=torch.bfloat16, device="cuda")
    pitched[:, O:] = float("nan")                                 # beside the rows: must not be read into the sums
    pitched[:, :O] = dy.cuda()
    ref = dy.double().t() @ x
    tol = (T + 8) * U * (dy.double().abs().t() @ x.abs())
    a = elmo.ckpt8_weight_grad(pitched[:, :O], codes, scales)
    off = (a.cpu().double() - ref).abs()
    assert bool((off <= tol).all()), (off / tol.clamp(min=1e-300)).max()
    b = elmo.ckpt8_weight_grad(dy.contiguous().cuda(), codes, scales)
    assert torch.equal(a, b)                                      # the pitch changes nothing, and it repeats
    base = torch.randn((O, D), generator=g).cuda()
    c = elmo.ckpt8_weight_grad(dy.contiguous().cuda(), codes, scales, out=base.clone(), accumulate=True)
    off = (c.cpu().double() - base.cpu().double() - ref).abs()
    assert bool((off <= tol + 8 * U * (base.cpu().double().abs() + ref.abs())).all())


def test_weight_gradient_of_one_hot_tokens(elmo):
    """dy with a single 1 per row picks rows of x exactly: every index of both operands is named."""
    T, O, D = 130, 136, 288
    codes, scales, x = _saved(T, D, 4)
    dy = torch.zeros((T, O), dtype=torch.bfloat16)
    at = torch.randperm(O, generator=torch.Generator().manual_seed(3))[:T]
    dy[torch.arange(T), at] = 1.0
    want = torch.zeros((O, D), dtype=torch.float64)
    want[at] = x
    assert torch.equal(elmo.ckpt8_weight_grad(dy.cuda(), codes, scales).cpu().double(), want)


def test_linear_layer_against_differences(elmo):
    """loss = sum(c * (x' W^T)) with the saved input x': dW is its gradient; and through silu's
    checkpoint, z -> sum(c * silu(z')): both against differences of float64 values."""
    T, O, D = 6, 16, 32
    x = _x(T, D, torch.float32, 9)
    codes, scales, _ = elmo.ckpt8_save(x)
    kept = elmo.ckpt8_load(codes, scales, dtype=torch.float32).cpu().double()
    c = torch.randn((T, O), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    dw = elmo.ckpt8_weight_grad(c.cuda(), codes, scales).cpu().double()
    W = torch.randn((O, D), generator=torch.Generator().manual_seed(5)).double()
    h = 2.0**-10
    for o, d in ((0, 0), (3, 31), (15, 7), (8, 16)):
        E = torch.zeros_like(W)
        E[o, d] = h
        ref = ((c.double() * (kept @ (W + E).t())).sum() - (c.double() * (kept @ (W - E).t())).sum()) / (2 * h)
        assert abs(float(dw[o, d] - ref)) < 1e-5 * float((c.double().abs().t() @ kept.abs())[o, d]) + 1e-9


def test_nan_codes_and_scales_reach_their_outputs_only(elmo):
    T, O, D = 40, 16, 64
    codes, scales, _ = _saved(T, D, 1)
    dy = torch.ones((T, O), dtype=torch.bfloat16, device="cuda")
    codes[7, 3] = 0x7F
    scales[9, 1] = 255
    bad = elmo.ckpt8_weight_grad(dy, codes, scales).isnan()
    want = torch.zeros((O, D), dtype=torch.bool, device="cuda")
    want[:, 3] = True
    want[:, 32:] = True
    assert torch.equal(bad, want)


def test_other_stream_and_empty(elmo):
    x = _x(100, 256, torch.bfloat16, 1)
    dy = _x(100, 64, torch.bfloat16, 2)
    codes, scales, y = elmo.ckpt8_save(x, act="gelu")
    dw = elmo.ckpt8_weight_grad(dy, codes, scales)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c2, s2, y2 = elmo.ckpt8_save(x, act="gelu")
        dw2 = elmo.ckpt8_weight_grad(dy, c2, s2)
    torch.cuda.synchronize()
    assert torch.equal(codes, c2) and torch.equal(scales, s2) and torch.equal(y, y2) and torch.equal(dw, dw2)
    codes, scales, y = elmo.ckpt8_save(x[:0], act="relu")
    assert codes.shape == (0, 256) and scales.shape == (0, 8) and y.shape == (0, 256)
    assert elmo.ckpt8_load(codes, scales).shape == (0, 256)
    assert bool((elmo.ckpt8_weight_grad(dy[:0], codes, scales) == 0).all())
    keep = torch.full((64, 256), 3.0, device="cuda")
    assert bool((elmo.ckpt8_weight_grad(dy[:0], codes, scales, out=keep, accumulate=True) == 3).all())


def test_refusals(elmo):
    x = _x(4, 64, torch.bfloat16, 1)
    codes, scales, _ = elmo.ckpt8_save(x)
    with pytest.raises(elmo.ElmoError):
        elmo.ckpt8_save(_x(4, 48, torch.bfloat16, 1))             # D % 32
    with pytest.raises(elmo.ElmoError):
        elmo.ckpt8_save(_x(4, 64, torch.bfloat16, 1, pad=4))      # rows not 16-byte aligned
    with pytest.raises(TypeError):
        elmo.ckpt8_save(x.double())
    with pytest.raises(ValueError):
        elmo.ckpt8_save(x, act="tanh")
    with pytest.raises(ValueError):
        elmo.ckpt8_load(codes, scales[:, :1])
    with pytest.raises(elmo.ElmoError):
        elmo.ckpt8_act_grad(x, codes, scales, None)
    with pytest.raises(ValueError):
        elmo.ckpt8_act_grad(x[:3], codes, scales, "relu")
    with pytest.raises(ValueError):
        elmo.ckpt8_weight_grad(x[:3], codes, scales)
    with pytest.raises(ValueError):
        elmo.ckpt8_weight_grad(x.float(), codes, scales)
    with pytest.raises(elmo.ElmoError):
        elmo.ckpt8_weight_grad(_x(4, 12, torch.bfloat16, 1), codes, scales)
    with pytest.raises(ValueError):
        elmo.ckpt8_weight_grad(x, codes, scales, accumulate=True)


def test_weight_grad_workspace_is_device_bytes(elmo):
    """A workspace on the host, of another type or strided is refused before its address is used."""
    codes, scales, _ = elmo.ckpt8_save(_x(600, 64, torch.bfloat16, 1))
    dy = _x(600, 64, torch.bfloat16, 2)
    want = elmo.ckpt8_weight_grad(dy, codes, scales)
    need = 1 << 21
    for bad in (torch.zeros(need, dtype=torch.uint8), torch.zeros(need, dtype=torch.float32, device="cuda"),
                torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            elmo.ckpt8_weight_grad(dy, codes, scales, workspace=bad)
    fine = torch.zeros(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(elmo.ckpt8_weight_grad(dy, codes, scales, workspace=fine), want)


@pytest.mark.parametrize("lo,hi", [(-13, -10), (-10, -9), (-9, -7), (-7, -5), (-5, -3), (-3, 0), (0, 3), (3, 14)])
def test_activations_over_their_ranges(elmo, lo, hi):
    """FP32 silu and gelu of four million values each: within the bounds above everywhere, their tails included."""
    g = torch.Generator(device="cuda").manual_seed(lo + 100)
    x = (torch.rand((1024, 4096), generator=g, device="cuda", dtype=torch.float64) * (hi - lo) + lo).float()
    for act in ("silu", "gelu"):
        codes, scales, y = elmo.ckpt8_save(x, act=act)
        for got, at, part in ((y, x.double(), 0),
                              (elmo.ckpt8_act_grad(torch.ones_like(x), codes, scales, act),
                               elmo.ckpt8_load(codes, scales, dtype=torch.float32).double(), 1)):
            v = _act64(at, act)
            ref, tol = v[part], v[part + 2]
            off = (got.double() - ref).abs()
            over = off / (tol + U * ref.abs() + TINY[torch.float32])
            assert bool((over <= 1).all()), f"{act} {'slope' if part else 'value'}: {over.max():.3f} of the tolerance at {at.flatten()[int(over.argmax())]}"
