"""Operators of the compiled binding run on their tensors' device, whichever is the current one, and refuse tensors of two."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def calls(ops, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = torch.randn(5, 288, generator=g, device=dev).to(torch.bfloat16)
    wt = (0.1 * torch.randn(1, 288, 288, generator=g, device=dev)).to(torch.bfloat16)
    with torch.cuda.device(dev):  # the weights are packed on their device
        w, ws, _ = ops.mxfp4_quantize_weights(wt)
    for quantize, linear, norm in ((ops.mxfp8_quantize, ops.mxfp8_linear, ops.moe_norm_in_mxfp8),
                                   (ops.mxfp4_quantize, ops.mxfp4_linear, ops.moe_norm_in)):
        c, s = quantize(x)
        yield from (c, s, linear(c, s, w[0], ws[0], 288), linear(c, s, w[0], ws[0], 288, y=torch.empty_like(x)))
        n = norm(x, x[0])
        yield n[0] if isinstance(n, tuple) else n


def test_tensors_of_another_device(ops):
    want = [t.cpu() for t in calls(ops, "cuda:0")]
    with torch.cuda.device(0):
        got = list(calls(ops, "cuda:1"))
        assert torch.cuda.current_device() == 0
    assert all(t.device.index == 1 for t in got)
    assert all(torch.equal(t.cpu(), w) for t, w in zip(got, want))


def test_tensors_of_two_devices_are_refused(ops):
    x = torch.zeros((4, 288), dtype=torch.bfloat16, device="cuda:0")
    codes = torch.zeros((4, 512), dtype=torch.uint8, device="cuda:1")
    with pytest.raises(ValueError, match="codes must be on cuda:0 with the other tensors, got cuda:1"):
        ops.mxfp8_quantize(x, codes=codes)
    with pytest.raises(ValueError, match="w must be on cuda:0"):
        ops.moe_norm_in_mxfp8(x, x[0].to("cuda:1"))
