"""Shapes of the layer that tests/test_gpu_mx8_layer.py leaves out, against the same oracle."""

import pytest
import torch

from test_gpu_mx8_layer import test_layer as check_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 64, 8192), (3, 4, 1, 64, 11264), (1, 2, 2, 96, 12320)])
def test_layer_of_few_pairs_in_shared_products(ops, T, E, k, H, I):
    """Up to three pairs whose products several workgroups share: the smallest LDS, all of it the waves' sums."""
    check_layer(ops, T, E, k, H, I)
