"""8-bit integer products of up to 32 rows over so many labels that a block shares its rows in LDS: features in one
panel of 1,024 and in several, steps that do not fill a batch, a last block with few labels. Whole sums on the device
in float64 (exact), tolerances as in the other tests of these products: 3 u + half a unit of the type, relative."""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,L,D", [(1, 65537, 128), (16, 66001, 320), (17, 65600, 192), (32, 65537, 1024), (5, 262301, 1088),
                                   (20, 262145, 2112), (16, 262273, 1536)])
def test_shared_rows(N, L, D, out):
    import precision_label_chunk_amd as elmo
    g = torch.Generator(device="cuda").manual_seed(N + D)
    X = torch.randint(-128, 128, (N, D), generator=g, device="cuda", dtype=torch.int8)
    W = torch.randint(-128, 128, (L, D), generator=g, device="cuda", dtype=torch.int8)
    sx, sw = torch.rand(N, generator=g, device="cuda") + 0.01, torch.rand(L, generator=g, device="cuda") * 1e-3
    print(f"  i8_matmul {N} x {L} x {D} {out}", flush=True)
    buf = torch.full((N, L + 3), 7.0, device="cuda", dtype=out)
    y = elmo.i8_matmul(X, sx, W, sw, out=buf[:, :L])
    step = 1 << 15
    for a in range(0, L, step):
        want = (X.double() @ W[a:a + step].double().t().contiguous()) * sx.double()[:, None] * sw[a:a + step].double()
        tol = want.abs() * (3 * 2.0**-24 + HALF[out] * (1 + 2.0**-22)) + (2.0**-25 if out == torch.float16 else 0.0)
        assert bool(((y[:, a:a + step].double() - want).abs() <= tol).all())
    assert bool((buf[:, L:] == 7.0).all())
