"""Log probabilities from features over more labels than one piece of the gradient may hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_labels_than_a_piece_holds():
    """4.5M labels, two rows: the library's pieces end at 2^22 labels. Sums over 4.5M labels of 32 features in float64 on
    the device, a part of the labels at a time; tolerances as a multiple of the unit roundings: G is held to
    2^-8, its sums' own error is below 2^-9 of that here."""
    import precision_label_chunk_amd as elmo
    N, V, D = 2, 4_500_000, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn((V, D), generator=g, device="cuda").to(torch.bfloat16)
    X = torch.randn((N, D), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([[V - 1], [(1 << 22) + 5]], device="cuda", dtype=torch.int32)
    r = elmo.linear_logprobs(X, W, ids)
    dx, dw = elmo.linear_logprobs_backward(X, W, ids, r, torch.full((N, 1), -1.0, device="cuda"),
                                           dx=torch.empty((N, D), device="cuda"), dw=torch.empty((V, D), device="cuda"))
    z = X.double() @ W.double().t()
    lse = torch.logsumexp(z, 1)
    assert float((r.row_max.double() + r.log_sum.double() - lse).abs().max()) < 1e-4
    assert float((r.logp.double() - (z.gather(1, ids.long()) - lse[:, None])).abs().max()) < 1e-4
    G = (z - lse[:, None]).exp()
    G.scatter_add_(1, ids.long(), torch.full((N, 1), -1.0, device="cuda", dtype=torch.float64))
    tol = 2.0**-8 * 1.1
    assert bool(((dw.double() - G.t() @ X.double()).abs() <= tol * (G.abs().t() @ X.double().abs()) + 1e-12).all())
    assert bool(((dx.double() - G @ W.double()).abs() <= tol * (G.abs() @ W.double().abs())).all())
