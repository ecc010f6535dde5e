"""Dropout's index of the first element: where the last index lies next to 2^64 the call is refused on the host (no GPU). The
kernel counts the generator's blocks by rounding the end up to 8, which wraps there, and would not end."""
import ctypes

import pytest
import torch

from test_abi_more import L  # noqa: F401

P, O = ctypes.c_void_p(4096), ctypes.c_void_p(65536)


def _call(L, first, T=4, D=8):  # noqa: F811
    return L.elmo_dropout(P, 0, T, D, D, None, 0, 0.5, 1, 2, None, first, O, D, None)


@pytest.mark.parametrize("T,D", [(1, 1), (4, 8), (1, 32), (3, 5), (2**31 - 1, 2**31 - 1)])
def test_last_indices_are_refused(L, T, D):  # noqa: F811
    n = T * D
    for end in range(2**64 - 7, 2**64 + 2):
        if end - n < 2**64:
            assert _call(L, end - n, T, D) == -1, (T, D, end)
    assert _call(L, 2**64 - 1, T, D) == -1
    assert _call(L, 2**64 - 8, T=0, D=D) == 0


def test_negative_index_is_refused():
    """A negative index does not stand for one next to 2^64."""
    import precision_label_chunk_amd as elmo
    for first in (-1, -2, -33, 2**64):
        with pytest.raises(ValueError, match="first"):
            elmo.dropout(torch.zeros(4, 8), 0.5, 1, first=first)
        with pytest.raises(ValueError, match="first"):
            elmo.dropout_backward(torch.zeros(4, 8), 0.5, 1, first=first)
