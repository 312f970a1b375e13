"""Calls of the training pass's operators that are refused on the host, with or without a GPU."""
import pytest


@pytest.fixture(scope="module")
def moe():
    from nvfp4_mixture_experts_softmax_gb300 import _build
    _build.build()
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


P = 4096   # a non-null, aligned address that no rejected call reads


@pytest.mark.parametrize("k", [1, 2])
def test_rows_gradient_in_the_place_of_dy(moe, k):
    """drows may take the place of rows, which each warp reads where it writes; not that of dy, which others still read."""
    assert moe.lib().moe_combine_rows_backward(P, 2 * P, P, P, 4, k, 64, 4 * k, 0, P, P, None) == -1
