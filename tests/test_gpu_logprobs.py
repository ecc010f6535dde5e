"""Log probabilities of given tokens, entropy, top alternatives and their gradient against a plain
float64 implementation on the CPU.

Tolerances (u = 2^-24). A lane adds at most c = ceil(V / 256) + 24 terms in a row (24 for the joins
after it), so sums of non-negative terms are off by at most c u relative. Each term e^(z - m) carries
the rounding of z - m, of its product with log2 e and of log2 e itself, together at most 3 |y| u in
the exponent y = (z - m) log2 e, and 2 ulp of the exponential; weighted by the terms themselves the
mean of |y| is at most log2 V + 2. So log s is off by R = (c + 3 (log2 V + 2) + 8) u absolute, logp
by R + 4 u |logp|, the entropy by R (2 + H) + 4 u H. p carries R + (3 |y| + 8) u relative."""
import itertools
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
UNIT = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 2.0**-149, torch.bfloat16: 2.0**-133, torch.float16: 2.0**-24}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def elmo():
    import precision_label_chunk_amd as m
    m.lib()
    return m


def _R(V):
    return (V / 256 + 25 + 3 * (math.log2(V) + 2) + 8) * U


def _plain(Z, ids, k):
    """float64: (logp, entropy, row_max, log_sum, top_idx, top_logp), with the empty row's values."""
    z = Z.detach().cpu().double()
    m = z.max(dim=1, keepdim=True).values
    empty = m == -math.inf
    y = torch.where(empty, torch.full_like(z, -math.inf), z - m)
    e = y.exp()
    s = e.sum(1, keepdim=True)
    logs = torch.where(empty, torch.zeros_like(s), s.log())
    H = logs - torch.where(e > 0, e * y, torch.zeros_like(e)).sum(1, keepdim=True) / torch.where(empty, torch.ones_like(s), s)
    lp = y - logs
    i = ids.cpu().long()
    logp = torch.where(i < 0, torch.zeros(i.shape, dtype=torch.float64), lp.gather(1, i.clamp(min=0)))
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    return logp, H[:, 0], m[:, 0], logs[:, 0], order, lp.gather(1, order)


def _close(got, ref, tol, what):
    got, ref = got.cpu().double(), ref.double()
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(ref)
    same = (got == ref) | (got.isnan() & ref.isnan())
    off = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    assert bool((same | (off <= tol)).all()), f"{what}: off by {off.max():.3e}, over {(off / tol).max():.3g} of the tolerance"


def _rows(N, V, dtype, seed, pad=0, shift=0, scale=3.0):
    """Logits as a view into a wider buffer, `shift` elements in, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn(N * (V + pad) + shift, generator=g) * scale).to(dtype).cuda()
    return buf[shift:].view(N, V + pad)[:, :V]


def _ids(N, V, M, seed):
    g = torch.Generator().manual_seed(seed + 1)
    ids = torch.randint(0, V, (N, M), generator=g, dtype=torch.int32)
    if M > 1:
        ids[:, 1:][torch.rand((N, M - 1), generator=g) < 0.3] = -1
    return ids.cuda()


def _check(elmo, Z, ids, k):
    V = Z.shape[1]
    print(f"  logprobs {tuple(Z.shape)} {Z.dtype} stride {Z.stride(0)} k={k}", flush=True)
    r = elmo.logprobs(Z, ids, k=k)
    logp, H, m, logs, order, top = _plain(Z, ids, k)
    R = _R(V)
    _close(r.row_max, m, 0.0, "row_max")
    _close(r.log_sum, logs, R, "log_sum")
    _close(r.logp, logp, R + 4 * U * logp.abs(), "logp")
    _close(r.entropy, H, R * (2 + H) + 4 * U * H, "entropy")
    if k:
        assert torch.equal(r.top_idx.cpu().long(), order)
        _close(r.top_logp, top, R + 4 * U * top.abs(), "top_logp")
    else:
        assert r.top_idx is None and r.top_logp is None
    return r


SHAPES = [(1, 1, 1), (3, 2, 2), (2, 7, 3), (5, 31, 31), (4, 513, 64), (3, 4097, 20), (300, 1000, 5), (2, 100003, 20),
          (1, 300000, 64), (37, 20011, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,k", SHAPES)
def test_logprobs(elmo, N, V, k, dtype):
    _check(elmo, _rows(N, V, dtype, V), _ids(N, V, 1, V), k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift,M,k", [(1, 0, 3, 0), (5, 1, 0, 7), (3, 3, 64, 64), (64, 0, 8, 0), (0, 7, 2, 5)])
def test_row_pitch_alignment_and_given_tokens(elmo, pad, shift, M, k, dtype):
    for V in (1003, 9000):
        Z = _rows(7, V, dtype, pad + V, pad=pad, shift=shift)
        _check(elmo, Z, _ids(7, V, M, pad), k)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_rows(elmo, dtype):
    """Rows with masked tokens, with one token left, with none, and masked by the type's lowest value."""
    V = 6001
    Z = _rows(6, V, dtype, 11)
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(4)
    Z[0][(torch.rand(V, generator=g) < 0.9).cuda()] = -math.inf
    Z[1] = -math.inf
    Z[1, 4444] = 2.5
    Z[2] = -math.inf
    Z[3] = low
    Z[4] = low
    Z[4, 17] = -1.0
    r = _check(elmo, Z, _ids(6, V, 3, 5), 20)
    assert r.entropy[2] == 0 and r.log_sum[2] == 0 and r.row_max[2] == -math.inf
    assert torch.equal(r.top_idx[2].cpu(), torch.arange(20, dtype=torch.int32)) and bool((r.top_logp[2] == -math.inf).all())
    assert abs(float(r.log_sum[3]) - math.log(V)) < _R(V)        # equal logits of any size: log V stays


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [1, 5, 64])
def test_ties_and_orders(elmo, dtype, k):
    """Equal logits go to the smallest token; rows in rising, falling and constant order."""
    V = 20000
    g = torch.Generator().manual_seed(k)
    rows = [torch.randint(0, 3, (V,), generator=g).float(), torch.zeros(V), torch.arange(V).float() / 16,
            -torch.arange(V).float() / 16, torch.cat([torch.full((V // 2,), -math.inf), torch.ones(V // 2)]),
            torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0), (torch.arange(V) % 97).float(),
            torch.cat([torch.full((V - 3,), -math.inf), torch.tensor([1.0, 2.0, 2.0])])]
    _check(elmo, torch.stack(rows).to(dtype).cuda(), _ids(len(rows), V, 1, k), k)


def test_nan_and_infinity(elmo):
    V = 5000
    for at in (0, 77, V - 1):
        Z = _rows(4, V, torch.float32, 8)
        Z[0, at] = math.nan
        Z[1, at] = math.inf
        Z[2] = math.nan
        ids = _ids(4, V, 2, 1)
        ids[:, 0] = (at + 1) % V
        r = elmo.logprobs(Z, ids, k=3)
        for n in (0, 1, 2):
            assert r.logp[n, 0].isnan() and r.entropy[n].isnan() and r.log_sum[n].isnan() and bool(r.top_logp[n].isnan().all())
        want = torch.sort(torch.nan_to_num(Z[0], nan=-math.inf), descending=True, stable=True).indices[:3]
        assert torch.equal(r.top_idx[0].long(), want)
        assert r.top_idx[1, 0] == at and r.row_max[1] == math.inf
        assert r.top_idx[2].tolist() == [0, 1, 2]
        assert bool(torch.isfinite(r.logp[3]).all())              # other rows are untouched
        dz = elmo.logprobs_backward(Z, ids, r, torch.ones_like(r.logp), dentropy=torch.ones(4, device="cuda"))
        assert bool(dz[:3].isnan().all()) and bool(torch.isfinite(dz[3]).all())


def test_nan_logits_rank_last(elmo):
    Z = torch.full((1, 3000), math.nan, device="cuda")
    Z[0, 2000:2003] = torch.tensor([1.0, -math.inf, 5.0], device="cuda")
    assert elmo.logprobs(Z, k=6).top_idx.tolist() == [[2002, 2000, 2001, 0, 1, 2]]


def test_token_out_of_range_is_nan(elmo):
    Z = _rows(2, 100, torch.float32, 3)
    ids = torch.tensor([[5, 100], [-1, -7]], dtype=torch.int32, device="cuda")
    r = elmo.logprobs(Z, ids)
    assert torch.isfinite(r.logp[0, 0]) and r.logp[0, 1].isnan()
    assert r.logp[1].tolist() == [0.0, 0.0]
    dz = elmo.logprobs_backward(Z, ids, r, torch.ones((2, 2), device="cuda"))
    assert bool(dz[0].isnan().all()) and bool((dz[1] == 0).all())


# ---- gradient --------------------------------------------------------------------------------------
def _plain_grad(Z, ids, dlogp, dH, dL):
    z = Z.detach().cpu().double()
    logp, H, m, logs, _, _ = _plain(Z, ids, 0)
    empty = (m == -math.inf)[:, None]
    lp = torch.where(empty, torch.full_like(z, -math.inf), z - m[:, None]) - logs[:, None]
    p = lp.exp()
    i = ids.cpu().long()
    g = torch.where(i < 0, torch.zeros(i.shape, dtype=torch.float64), dlogp.cpu().double())
    hot = torch.zeros_like(z).scatter_add_(1, i.clamp(min=0), g)
    hot_abs = torch.zeros_like(z).scatter_add_(1, i.clamp(min=0), g.abs())
    lps = torch.where(p > 0, lp, torch.zeros_like(lp))
    gh = dH.cpu().double()[:, None] if dH is not None else torch.zeros((z.shape[0], 1), dtype=torch.float64)
    gl = dL.cpu().double()[:, None] if dL is not None else torch.zeros((z.shape[0], 1), dtype=torch.float64)
    dz = torch.where(empty, torch.zeros_like(z), p * (gl - g.sum(1, keepdim=True) - gh * (lps + H[:, None])) + hot)
    size = p * (gl.abs() + g.abs().sum(1, keepdim=True) + gh.abs() * (lps.abs() + H[:, None])) + hot_abs
    return dz, size, p * lps.abs() * (size / p.clamp(min=1e-300)).clamp(max=1e30)


def _check_grad(elmo, Z, ids, seed=0, dH=True, dL=False, in_place=False, out=None):
    N, V = Z.shape
    g = torch.Generator().manual_seed(seed + 99)
    dlogp = torch.randn(ids.shape, generator=g).cuda()
    dh = torch.randn(N, generator=g).cuda() if dH else None
    dl = torch.randn(N, generator=g).cuda() if dL else None
    print(f"  grad {tuple(Z.shape)} {Z.dtype} stride {Z.stride(0)} M={ids.shape[1]}", flush=True)
    r = elmo.logprobs(Z, ids)
    ref, size, spread = _plain_grad(Z, ids, dlogp, dh, dl)
    got = elmo.logprobs_backward(Z, ids, r, dlogp, dentropy=dh, dlse=dl, out=Z if in_place else out)
    if in_place:
        assert got.data_ptr() == Z.data_ptr()
    # p off by R + (3 |y| + 8) u relative, its factor by R (entropy) and the roundings of M + 4 terms
    tol = 2 * (_R(V) + (8 + ids.shape[1] + 4) * U) * size + 5 * U * spread + UNIT[Z.dtype] * ref.abs() + TINY[Z.dtype]
    _close(got, ref, tol, "dZ")
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,M", [(1, 1, 1), (3, 2, 1), (2, 7, 4), (4, 513, 1), (3, 4097, 64), (300, 1000, 2), (2, 100003, 8)])
def test_gradient(elmo, N, V, M, dtype):
    _check_grad(elmo, _rows(N, V, dtype, V + 1), _ids(N, V, M, V), seed=V)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dH,dL", list(itertools.product([False, True], repeat=2)))
def test_gradient_parts_strides_and_in_place(elmo, dtype, dH, dL):
    V = 2003
    for pad, shift in ((0, 0), (1, 0), (5, 3)):
        ids = _ids(5, V, 6, pad)
        ids[0] = ids[0, 0]                                        # one token given six times
        ids[1, 1], ids[1, 3] = ids[1, 0], ids[1, 0]
        _check_grad(elmo, _rows(5, V, dtype, 21, pad, shift), ids, dH=dH, dL=dL)
        _check_grad(elmo, _rows(5, V, dtype, 22, pad, shift), ids, dH=dH, dL=dL, in_place=True)
        wide = torch.zeros((5, V + 9), dtype=dtype, device="cuda")
        _check_grad(elmo, _rows(5, V, dtype, 23, pad, shift), ids, dH=dH, dL=dL, out=wide[:, 2:2 + V])
        assert bool((wide[:, :2] == 0).all()) and bool((wide[:, 2 + V:] == 0).all())   # nothing beside the rows


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_masked_rows(elmo, dtype):
    V = 4100
    Z = _rows(4, V, dtype, 31)
    Z[0, ::2] = -math.inf
    Z[1] = -math.inf
    Z[2] = torch.finfo(dtype).min
    Z[3] = -math.inf
    Z[3, 5] = 1.0
    ids = _ids(4, V, 2, 6)
    ids[0, 0] = 2                                                 # a given token that is masked: p = 0
    got = _check_grad(elmo, Z, ids, dL=True)
    assert bool((got[1] == 0).all())


def test_gradient_against_differences(elmo):
    """Central differences of the float64 value sum(g logp) + sum(gH H) + sum(gL lse)."""
    N, V, M = 3, 97, 3
    Z, ids = _rows(N, V, torch.float32, 5, scale=1.5), _ids(N, V, M, 5)
    g = torch.Generator().manual_seed(77)
    dlogp, dh, dl = torch.randn((N, M), generator=g), torch.randn(N, generator=g), torch.randn(N, generator=g)
    got = elmo.logprobs_backward(Z, ids, elmo.logprobs(Z, ids), dlogp.cuda(), dh.cuda(), dl.cuda()).cpu().double()

    def value(z):
        logp, H, m, logs, _, _ = _plain(z, ids, 0)
        return (dlogp.double() * logp).sum(1) + dh.double() * H + dl.double() * (m + logs)

    z, h = Z.cpu().double(), 1e-4
    for v in range(V):
        d = torch.zeros_like(z)
        d[:, v] = h
        # the differences' own error: h^2 times the third derivative (a few units here) and 1e-16 / h
        ref = (value(z + d) - value(z - d)) / (2 * h)
        assert (got[:, v] - ref).abs().max() < 1e-5


def test_repeats_bit_for_bit_and_on_another_stream(elmo):
    Z, ids = _rows(6, 50021, torch.bfloat16, 9), _ids(6, 50021, 4, 9)
    a = elmo.logprobs(Z, ids, k=20)
    da = elmo.logprobs_backward(Z, ids, a, torch.ones_like(a.logp), dentropy=torch.ones(6, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = elmo.logprobs(Z, ids, k=20)
        db = elmo.logprobs_backward(Z, ids, b, torch.ones_like(b.logp), dentropy=torch.ones(6, device="cuda"))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert torch.equal(da, db)


def test_graph_replays(elmo):
    """Captured once, replayed with new logits and the program's own work in between."""
    Z, ids = _rows(2, 70001, torch.float32, 1), _ids(2, 70001, 2, 1)
    N, V = Z.shape
    ws = torch.empty(elmo.lib().elmo_logprobs_workspace_bytes(N, V, 9), dtype=torch.uint8, device="cuda")
    g1 = torch.randn((N, 2), device="cuda")
    elmo.logprobs(Z, ids, k=9, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = elmo.logprobs(Z, ids, k=9, workspace=ws)
        dz = elmo.logprobs_backward(Z, ids, r, g1)
    for seed in range(4):
        Z.copy_(_rows(N, V, torch.float32, 100 + seed))
        graph.replay()
        torch.cuda.synchronize()
        e = elmo.logprobs(Z, ids, k=9)
        for x, y in zip(r, e):
            assert torch.equal(x, y)
        assert torch.equal(dz, elmo.logprobs_backward(Z, ids, e, g1))


def test_empty_batch_and_refusals(elmo):
    Z = torch.zeros((0, 50), device="cuda")
    r = elmo.logprobs(Z, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), k=3)
    assert r.logp.shape == (0, 2) and r.top_idx.shape == (0, 3)
    Z = _rows(2, 50, torch.float32, 1)
    ids = _ids(2, 50, 1, 1)
    with pytest.raises(elmo.ElmoError):
        elmo.logprobs(Z, ids, k=51)
    with pytest.raises(elmo.ElmoError):
        elmo.logprobs(torch.zeros((2, 100), device="cuda"), k=65)
    with pytest.raises(elmo.ElmoError):
        elmo.logprobs(Z, torch.zeros((2, 65), dtype=torch.int32, device="cuda"))
    with pytest.raises(elmo.ElmoError):
        elmo.logprobs(Z[:1].expand(2, 50))                        # rows on top of each other
    with pytest.raises(TypeError):
        elmo.logprobs(Z.double())
    with pytest.raises(ValueError):
        elmo.logprobs(Z, ids.long())
    with pytest.raises(ValueError):
        elmo.logprobs(Z.t())                                      # elements of a row not adjacent
    with pytest.raises(ValueError):
        elmo.logprobs(Z.cpu())
    r = elmo.logprobs(Z, ids)
    with pytest.raises(ValueError):
        elmo.logprobs_backward(Z, ids, r, torch.zeros((2, 2), device="cuda"))
    with pytest.raises(ValueError):
        elmo.logprobs_backward(Z, ids, r, None)
    with pytest.raises(ValueError):
        elmo.logprobs_backward(Z, ids, r, r.logp, out=torch.zeros((2, 49), device="cuda"))


@pytest.mark.parametrize("dtype,bits,view", [(torch.float32, 0x7F800001, torch.int32), (torch.bfloat16, 0x7F81, torch.int16),
                                             (torch.float16, 0x7C01, torch.int16)])
@pytest.mark.parametrize("k", [4, 40])
def test_signalling_nan_logits_hide_no_alternative(elmo, dtype, bits, view, k):
    """Signalling NaNs beside the largest logits: the alternatives are those of the other tokens."""
    for V in (3000, 40000):
        g = torch.Generator().manual_seed(V)
        Z = (torch.randn(2, V, generator=g) * 3).to(dtype)
        bad = torch.zeros(2, V, dtype=torch.bool)
        best = Z.float().topk(k, dim=1).indices
        for n in range(2):
            for i in best[n].tolist():
                for j in (i - 1, i + 1, i ^ 4):
                    if 0 <= j < V and j not in best[n]:
                        bad[n, j] = True
        want = torch.sort(torch.where(bad, torch.full_like(Z, -math.inf), Z).float(), dim=1, descending=True, stable=True).indices[:, :k]
        raw = Z.view(view).clone()
        raw[bad] = bits
        r = elmo.logprobs(raw.view(dtype).cuda(), k=k)
        assert torch.equal(r.top_idx.cpu().long(), want)
        assert bool(r.entropy.isnan().all())


def test_workspace_is_device_bytes(elmo):
    """A workspace on the host, of another type or strided is refused before its address is used."""
    Z = torch.randn(2, 70000, device="cuda")
    want = elmo.logprobs(Z, k=3)
    need = 1 << 20
    for bad in (torch.zeros(need, dtype=torch.uint8), torch.zeros(need, dtype=torch.float32, device="cuda"),
                torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            elmo.logprobs(Z, k=3, workspace=bad)
    for fine in (torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.zeros(8, dtype=torch.uint8, device="cuda")):
        r = elmo.logprobs(Z, k=3, workspace=fine)
        assert torch.equal(r.entropy, want.entropy) and torch.equal(r.top_idx, want.top_idx)


@pytest.mark.parametrize("k", [0, 2])
def test_one_token_over_many_at_the_lowest_value(elmo, k):
    """1.5e9 tokens masked with the type's lowest value and one that is not: sums of more than 3.4e8
    equal terms meet a distance that binary32 does not hold. The token has all the probability."""
    V = 1_500_000_001
    Z = torch.full((1, V), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device="cuda")
    Z[0, V - 2] = 1.0
    ids = torch.tensor([[V - 2]], dtype=torch.int32, device="cuda")
    r = elmo.logprobs(Z, ids, k=k)
    assert r.row_max.item() == 1.0 and r.log_sum.item() == 0.0
    assert r.logp.item() == 0.0 and r.entropy.item() == 0.0
    if k:
        assert r.top_idx.cpu().tolist() == [[V - 2, 0]] and r.top_logp[0, 0].item() == 0.0


def test_more_rows_than_one_launch_holds(elmo):
    """2^24 + 5 rows: 256 threads each would be more than 2^32. Rows do not depend on each other, so
    every stretch of them equals its own call bit for bit, and the last ones the plain form."""
    N, V = (1 << 24) + 5, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    Z = torch.randn((N, V), device="cuda", generator=g).half()
    ids = torch.randint(0, V, (N, 1), device="cuda", generator=g, dtype=torch.int32)
    r = elmo.logprobs(Z, ids, k=2)
    d = torch.randn((N, 1), device="cuda", generator=g)
    dZ = elmo.logprobs_backward(Z, ids, r, d)
    for a, b in ((0, 1000), ((1 << 23) - 3, (1 << 23) + 3), ((1 << 24) - 2, N)):
        part = elmo.logprobs(Z[a:b], ids[a:b], k=2)
        for x, y in zip(r, part):
            assert torch.equal(x[a:b], y)
        assert torch.equal(dZ[a:b], elmo.logprobs_backward(Z[a:b], ids[a:b], part, d[a:b]))
    lp = Z[-7:].cpu().double().log_softmax(1)
    err = (r.logp[-7:].cpu().double() - lp.gather(1, ids[-7:].cpu().long())).abs().max()
    assert err <= _R(V) + 4 * U * lp.abs().max()


def test_ids_that_name_no_token_in_empty_and_nan_rows(elmo):
    """An id past the vocabulary gives NaN and a negative one 0 in any row; the gradient of a row without
    tokens is 0 whatever its ids, that of any other row with an id past the vocabulary NaN."""
    V = 1001
    Z = _rows(4, V, torch.float32, 6)
    Z[0], Z[1], Z[2, 5] = -math.inf, math.nan, math.inf
    ids = torch.tensor([[V, -1, 3]] * 4, dtype=torch.int32, device="cuda")
    r = elmo.logprobs(Z, ids, k=2)
    assert bool(r.logp[:, 0].isnan().all()) and bool((r.logp[:, 1] == 0).all())
    assert r.logp[0, 2] == -math.inf and bool(r.logp[1:3, 2].isnan().all()) and bool(torch.isfinite(r.logp[3, 2]))
    assert r.row_max[:3].tolist() == [-math.inf, -math.inf, math.inf]
    for dh in (None, torch.ones(4, device="cuda")):
        dz = elmo.logprobs_backward(Z, ids, r, torch.ones((4, 3), device="cuda"), dentropy=dh)
        assert bool((dz[0] == 0).all()) and bool(dz[1:].isnan().all())


def test_a_row_gives_the_same_alternatives_in_any_batch(elmo):
    """Rows are split differently in batches of different sizes: the alternatives stay, the sums within their bounds."""
    Z = _rows(600, 70001, torch.bfloat16, 12)
    r = elmo.logprobs(Z, k=20)
    for n in (0, 1, 599):
        one = elmo.logprobs(Z[n:n + 1], k=20)
        assert torch.equal(one.top_idx[0], r.top_idx[n]) and one.row_max[0] == r.row_max[n]
        assert abs(float(one.log_sum[0] - r.log_sum[n])) <= 2 * _R(70001)
