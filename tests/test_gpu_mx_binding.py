"""What the binding accepts and refuses of tensors on the device."""

import numpy as np
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


@pytest.mark.parametrize("flag", [1, np.True_, True])
def test_quantize_is_any_truth_value(ops, flag):
    x = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    want = ops.moe_norm_in(x, x[0], quantize=True)
    got = ops.moe_norm_in(x, x[0], quantize=flag)
    assert len(got) == 3 and all(torch.equal(a, b) for a, b in zip(got, want))
    assert len(ops.moe_norm_out(x, x, None, x[0], quantize=flag)) == 4
    with pytest.raises(ValueError, match="need w_next"):
        ops.moe_norm_out(x, x, quantize=flag)


@pytest.mark.parametrize("flag", [0, np.False_, False, None])
def test_quantize_is_any_false_value(ops, flag):
    x = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    assert torch.equal(ops.moe_norm_in(x, x[0], quantize=flag), ops.moe_norm_in(x, x[0]))


def test_combine_of_sizes_that_wrap(ops):
    """T * k and T * H beyond 64 bits are not taken for small numbers (nothing may be enqueued)."""
    po, ps = torch.zeros(8, 64, dtype=torch.float16, device="cuda"), torch.zeros(8, device="cuda")
    y = torch.zeros(8, 64, device="cuda")
    for T, k in ((1 << 62, 4), (1 << 62, 8), (1 << 58, 64)):
        with pytest.raises(ValueError, match="pair_out must be"):
            ops.moe_combine(po, ps, T, k, y=y)
    with pytest.raises(ValueError, match="y must hold"):
        ops.moe_combine(po, ps, 1 << 62, 0, y=y)
    with pytest.raises(ops.MoEError, match="MOE_ERR_SHAPE"):
        ops.moe_combine(po, ps, -1, 2, y=y)
