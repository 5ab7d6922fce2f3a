"""The activations of mxfp8_linear on exactly known sums: with x = 0 the bias is z, so every BF16 value is an argument.

Bounds, u = 2^-24 (FP32's rounding): ReLU exact.  SiLU and the tanh form, from the hardware's exponential and reciprocal (2 u each)
on an argument rounded a few times: (8 + 4 |z| + 4 |z|^3) 2 u of the result (the cube for the tanh form only).  GELU by erf: 16 u of
the result: 2.7e-8 of the fit is u / 2, its reciprocal's argument and value 3 u (the tail goes with less than its first power), eight
steps of Horner's rule whose later terms are smaller 3 u, the exponential 2 u, the exponent's parts u, and five products u each.
BF16 results add half a step, 2^-8; results of less than 1e-36 may be zero."""

import math

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, to_np
from workloads import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def arguments():
    """Every BF16 value of 2^-60 to 64 by magnitude, and zeros."""
    bits = np.arange(65536, dtype=np.uint16)
    with np.errstate(invalid="ignore"):
        v = gen.bf16_bits_to_f32(bits).astype(np.float64)
        return bits[(np.abs(v) <= 64) & ((np.abs(v) >= 2.0 ** -60) | (v == 0))]


def reference(name, z):
    m = np.abs(z)
    if name == "relu":
        return np.maximum(z, 0.0), 0.0
    if name == "silu":
        return z / (1.0 + np.exp(-z)), (8 + 4 * m) * 2 * U
    if name == "gelu":
        return 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2.0)), 16 * U
    w = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    return z / (1.0 + np.exp(np.minimum(-2.0 * w, 700.0))), (8 + 4 * m + 4 * m ** 3) * 2 * U


# few columns: streamed; many: tiles, of which the first token's columns are looked at
@pytest.mark.parametrize("T,parts", [(1, 2), (5, 4), (40, 4), (130, 1), (300, 1)])
@pytest.mark.parametrize("name", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activation_of_every_value(T, parts, name):
    from nvfp4_w4a4_mixture_amd import ops

    bits = arguments()
    for b in np.array_split(bits, parts):
        N = b.size
        wc, ws, _ = ops.mxfp4_quantize_weights(torch.ones((1, N, 32), dtype=torch.bfloat16, device="cuda"))
        codes, scales = ops.mxfp8_quantize(torch.zeros((T, 32), dtype=torch.bfloat16, device="cuda"))
        z = gen.bf16_bits_to_f32(b).astype(np.float64)
        ref, rel = reference(name, z)
        for dtype in (torch.float32, torch.bfloat16):
            y = ops.mxfp8_linear(codes, scales, wc[0], ws[0], N, dtype, bias=dev_bf16(b), activation=name)
            assert bool((y == y[:1]).all())
            got = to_np(y[0].float()).astype(np.float64)
            bound = rel * np.abs(ref)
            if dtype == torch.bfloat16:
                bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
            worst = np.max((np.abs(got - ref) - 1e-36) / np.maximum(bound, 1e-300))
            print(f"  {name} {dtype} {worst:.3f}", flush=True)
            assert (np.abs(got - ref) <= bound + 1e-36).all()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_gelu_of_extremes(T):
    """Large arguments, infinity and NaN."""
    from nvfp4_w4a4_mixture_amd import ops

    b = torch.tensor([1e30, float("inf"), float("nan"), -1e30, -20.0, 0.0, -0.0, 3e38], device="cuda").to(torch.bfloat16)
    wc, ws, _ = ops.mxfp4_quantize_weights(torch.ones((1, 8, 32), dtype=torch.bfloat16, device="cuda"))
    codes, scales = ops.mxfp8_quantize(torch.zeros((T, 32), dtype=torch.bfloat16, device="cuda"))
    for name in ("gelu", "gelu_tanh"):
        y = ops.mxfp8_linear(codes, scales, wc[0], ws[0], 8, torch.float32, bias=b, activation=name)
        assert bool(y[:, 2].isnan().all()) and torch.equal(y[:, [0, 1, 7]], b[[0, 1, 7]].float().expand(T, 3))
        assert bool((y[:, 3:7] == 0).all())
