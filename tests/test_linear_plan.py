"""Which tile shape the gradient from features takes (no GPU): by the time each is expected to take, over many rows and labels
too."""
import pytest

from test_more_kernels import _shape, backward, record  # noqa: F401


@pytest.mark.parametrize("N,V", [(1024, 16384), (4096, 32003), (2698, 120686)])
def test_few_features_take_smaller_tiles(record, N, V):  # noqa: F811
    """A tile of few features is done with its products soon, and smaller ones overlap its results with others' products."""
    few, many = record([backward(1, N, V, 64), backward(1, N, V, 2048)])
    assert "4" not in {_shape(x[0]) for x in few[1] if "k_lin_products" in x[0]}
    assert {_shape(x[0]) for x in many[1] if "k_lin_products" in x[0]} == {"4"}
