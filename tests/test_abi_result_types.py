"""The workspace of the gradient from features by its results' types (no GPU): a query that tells them gives what the call
takes, one that does not gives enough for any."""
import ctypes

import pytest

from test_abi_more import L  # noqa: F401

P, O = ctypes.c_void_p(4096), ctypes.c_void_p(65536)
TYPES = (0, 1, 2)                            # FP32, BF16, FP16


@pytest.mark.parametrize("N,V,D,chunk", [(1, 100, 64, 0), (128, 5000, 96, 0), (129, 5000, 96, 256), (512, 1000, 256, 0),
                                         (4096, 131072, 768, 0), (5000, 300, 64, 0)])
def test_query(L, N, V, D, chunk):  # noqa: F811
    def size(dx, dw):
        return L.elmo_linear_logprobs_backward_workspace_bytes(N, V, D, 1, chunk, dx, dw)

    def call(dx, dw, wb):
        return L.elmo_linear_logprobs_backward(P, P, 1, N, V, D, D, D, P, 1, P, P, P, None, None if dx is None else O, dx or 0, D,
                                               None if dw is None else O, dw or 0, D, 0, chunk, P, wb, None)
    for dx in (None, *TYPES):
        for dw in (None, *TYPES):
            if dx is None and dw is None:
                continue
            need = size(0 if dx is None else 2 + dx, 0 if dw is None else 2 + dw)
            assert 0 < need <= size(0 if dx is None else 1, 0 if dw is None else 1)
            assert call(dx, dw, need - 1) == -4
    assert size(3, 3) == size(4, 4) == size(3, 4)
    assert size(1, 1) == size(9, -1) == max(size(2 + dx, 2 + dw) for dx in TYPES for dw in TYPES)
