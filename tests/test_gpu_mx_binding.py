"""What the binding accepts and refuses of tensors on the device."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def test_combine_into_a_given_y(ops):
    """A given y sets the result's type; one that the result does not fit is refused before anything is enqueued."""
    T, k, H = 5, 2, 96
    po, ps = torch.randn(T * k, H, device="cuda").to(torch.float16), torch.full((T * k,), 0.5, device="cuda")
    want = {d: ops.moe_combine(po, ps, T, k, d) for d in (torch.bfloat16, torch.float32)}
    for asked in want:
        for dtype in want:
            y = torch.full((T + 1, H), 7.0, dtype=dtype, device="cuda")
            got = ops.moe_combine(po, ps, T, k, asked, y=y)
            assert got.data_ptr() == y.data_ptr() and torch.equal(y[:T], want[dtype]) and bool((y[T] == 7).all())
    flat = torch.empty(T * H, device="cuda")
    ops.moe_combine(po, ps, T, k, y=flat)
    assert torch.equal(flat.view(T, H), want[torch.float32])

    def refused(kind, match, y, **kw):
        with pytest.raises(kind, match=match):
            ops.moe_combine(po, ps, T, k, y=y, **kw)

    refused(TypeError, "output type", torch.empty((T, H), dtype=torch.float16, device="cuda"))
    refused(TypeError, "output type", torch.empty((T, H), dtype=torch.int32, device="cuda"))
    refused(ValueError, "y must hold", torch.empty((T - 1, H), device="cuda"))
    refused(ValueError, "y must be contiguous", torch.empty((T, 2 * H), device="cuda")[:, :H])
    refused(ValueError, "GPU", torch.empty((T, H)))
    with pytest.raises(TypeError, match="output type"):
        ops.moe_combine(po, ps, T, k, torch.float16)
