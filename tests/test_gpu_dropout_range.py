"""Dropout at the largest indices that it takes."""
import pytest
import torch

from test_gpu_dropout import F32, _same, elmo, plain  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(1, 1), (1, 32), (4, 8), (3, 5), (37, 19)])
def test_largest_first(elmo, T, D):  # noqa: F811
    x = torch.randn((T, D), device="cuda")
    for end in (2**64 - 8, 2**64 - 9, 2**64 - 16):
        first = end - T * D
        print(f"  dropout {T} x {D} from {first}", flush=True)
        assert _same(elmo.dropout(x, 0.5, 9, 2, first=first), plain(x, 0.5, 9, 2, first=first)), (T, D, end)
    assert x.dtype == F32
