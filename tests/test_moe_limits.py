"""Sizes that the calls of include/gmm_moe.h refuse because a launch could not
hold them, on the CPU: every refusal comes before any launch."""
import pytest

import moe_grouped_gemm_gmm_amd as gmm
from test_moe_boundary import SHAPE, WORKSPACE, linear_bwd


@pytest.fixture(scope="module")
def lib():
    return gmm.load_library()


# The bias gradient's second launch has a workgroup of 256 for every 64 columns
# of every group, however few rows there are: fewer than 2^24 of them.
@pytest.mark.parametrize("G,N", [(4096, 1 << 18), (4096, (1 << 18) + 64), (64, 1 << 24), (4096, 1 << 30)])
def test_bias_gradient_of_too_many_columns_is_refused(lib, G, N):
    for M in (0, 1):
        assert linear_bwd(lib, M=M, K=64, N=N, G=G, dx=0, dw=0) == SHAPE
        assert lib.gmm_last_error()


def test_the_largest_bias_gradient_is_not(lib):
    # without a workspace, which is asked for after the sizes
    assert linear_bwd(lib, M=1, K=64, N=(1 << 18) - 64, G=4096, dx=0, dw=0, ws=0) == WORKSPACE
    # the other gradients do not need that launch
    assert linear_bwd(lib, M=1, K=64, N=1 << 18, G=4096, dx=0, db=0, ws=0) == WORKSPACE
