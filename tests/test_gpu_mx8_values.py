"""Every BF16 value through the MXFP8 quantizer, under every distance to the largest value of its block that a normal block
scale reaches: by itself, and beside first elements of 1, 2, 4, 8 .. 2^18 times its size."""

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, to_np
from oracle import mx8
from workloads import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("times", [0, 0.5, 1, 2, 3, 4, 8, 16, 96, 256, 2.0 ** 10, 2.0 ** 14, 2.0 ** 16, 2.0 ** 18])
def test_every_bf16_value_beside_larger_ones(times):
    from nvfp4_w4a4_mixture_amd import ops

    bits = np.arange(65536, dtype=np.uint16)
    v = gen.bf16_bits_to_f32(bits).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        first = (np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0) * times).astype(np.float32)
    # BF16 by truncation: the oracle sees the same bits, so any rounding does
    fbits = (first.view(np.uint32) >> 16).astype(np.uint16)
    x = np.zeros((65536, 32), np.uint16)
    x[:, 0], x[:, 9] = fbits, bits
    codes, scales = ops.mxfp8_quantize(dev_bf16(x))
    oc, ob = mx8.quantize(gen.bf16_bits_to_f32(x).astype(np.float64))
    assert np.array_equal(to_np(scales)[:, :1], ob) and np.array_equal(to_np(codes)[:, :32], oc)
    share = float(((oc[:, 9] & 0x7F) > 0).mean())
    assert share > 0.9  # not a test of zero codes
