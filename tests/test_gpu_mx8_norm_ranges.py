"""The MXFP8 norms over the whole range of their rows' number."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def test_norm_of_the_most_rows(ops):
    """More rows than a launch of five waves each can have (2^32 work-items), of a width that takes five waves otherwise."""
    T, H = 13_421_773 + 5, 2080
    assert T * 320 > 2 ** 32 > T * 256
    if torch.cuda.mem_get_info()[0] < 120e9:
        pytest.skip("needs 120 GB of device memory")
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").zero_()
    at = [0, 1, T // 3, 13_421_771, 13_421_772, 13_421_773, T - 1]
    some = torch.randn(len(at), H, device="cuda").to(torch.bfloat16)
    for i, t in enumerate(at):
        x[t] = some[i]
    w = torch.randn(H, device="cuda").to(torch.bfloat16)
    want = ops.moe_norm_in_mxfp8(some, w, n=False)
    _, codes, scales = ops.moe_norm_in_mxfp8(x, w, n=False)
    for i, t in enumerate(at):
        assert torch.equal(codes[t], want[1][i]) and torch.equal(scales[t], want[2][i])
    assert not bool(codes[2:5].any()) and not bool(scales[T - 4: T - 1].any())
    del x, codes, scales
    torch.cuda.empty_cache()
