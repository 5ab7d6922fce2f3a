"""The MXFP8 norms over the whole range of their inputs' sizes and of their rows' number."""

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, say, to_np
from oracle import norm as onorm
from test_gpu_mx import bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def f64(t):
    return to_np(t.float()).astype(np.float64)


def near(got, ref):
    """Half a BF16 step, and FP32's roundings before it (tests/test_gpu_mx8.py)."""
    g = f64(got)
    step = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(np.abs(g), np.abs(ref)))[1], -125) - 8)
    assert np.isfinite(g).all()
    assert (np.abs(g - ref) <= step / 2 + 2.0 ** -22 * np.abs(ref)).all()


@pytest.mark.parametrize("T,H", [(2, 32), (3, 288), (1, 2080), (300, 4128), (1, 6144)])
@pytest.mark.parametrize("size", [2.0 ** -133, 2.0 ** -128, 2.0 ** -100, 2.0 ** 60, 2.0 ** 120])
def test_norms_of_any_size_without_eps(ops, T, H, size):
    """x / rms(x) does not depend on the rows' size: not where 1 / rms leaves FP32, nor where x is subnormal."""
    say(f"norms {T}x{H} of {size}")
    rng = np.random.default_rng(T + H)
    xv, xb = bf16(np.rint(rng.standard_normal((T, H)) * 8) * size)
    wv, wb = bf16(1 + 0.3 * rng.standard_normal(H))
    rv, rb = bf16(rng.standard_normal((T, H)))
    x, w, r = dev_bf16(xb), dev_bf16(wb), dev_bf16(rb)
    n, codes, scales = ops.moe_norm_in_mxfp8(x, w, 0.0)
    near(n, onorm.norm(xv, wv, 0.0))
    c, s = ops.mxfp8_quantize(n)
    assert torch.equal(codes, c) and torch.equal(scales, s)
    y32 = (xv * 0.37).astype(np.float32)  # FP32 subnormals too
    out = ops.moe_norm_out_mxfp8(torch.from_numpy(y32).cuda(), r, w, w, residual_scale=0.5, eps=0.0)[0]
    ref = onorm.residual(y32.astype(np.float64), rv, wv, None, 0.5, 0.0)
    half = np.ldexp(1.0, np.frexp(np.maximum(np.abs(f64(out)), np.abs(ref)))[1] - 9)
    assert (np.abs(f64(out) - ref) <= half + 2.0 ** -22 * (np.abs(ref) + np.abs(ref - rv))).all()


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
    assert not bool((codes[2:5] & 0x7F).any()) and not bool(scales[T - 4: T - 1].any())  # zeros of either sign
    del x, codes, scales
    torch.cuda.empty_cache()
