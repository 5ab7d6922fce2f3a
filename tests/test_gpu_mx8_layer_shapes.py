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


@pytest.mark.parametrize("T,E,k,H,I", [(16, 16, 4, 288, 1504), (16, 80, 8, 512, 512), (1, 40, 20, 64, 1056), (32, 30, 6, 96, 800)])
def test_layer_of_many_tiles(ops, T, E, k, H, I):
    """More than 512 tiles of h: a workgroup walks several, and loads ahead from one expert's into the next one's; ranked by
    gate_up and by a kernel of its own, in one operand and in two."""
    check_layer(ops, T, E, k, H, I)


@pytest.mark.parametrize("T,E,k,H,I", [(32, 32, 4, 64, 32), (8, 64, 8, 96, 64), (2, 128, 8, 64, 32), (16, 48, 4, 64, 32),
                                       (16, 64, 8, 96, 64), (1, 256, 8, 64, 32)])
def test_layer_where_the_ranking_changes(ops, T, E, k, H, I):
    """The most scores that gate_up ranks itself, and the fewest that a kernel before it does."""
    check_layer(ops, T, E, k, H, I)
