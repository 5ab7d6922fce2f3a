"""GPU parity of moe_norm_in and moe_norm_out against oracle/norm.py (float64).

Bounds: FP32 sums and products of H terms, (H + 16) u of each term's size with u = 2^-24, and one BF16 rounding,
half an ulp (2^-8 of the value, or half the smallest subnormal).  At most 1% of the results (and one more) may differ
from the correctly rounded value: FP32 noise of some 2^-21 against rounding intervals of 2^-8."""

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, say, to_np
from oracle import norm as onorm
from workloads import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def bf16(a):
    bits = gen.f32_to_bf16_bits(np.ascontiguousarray(a, dtype=np.float32))
    return gen.bf16_bits_to_f32(bits).astype(np.float64), bits


def values(t):
    return to_np(t.float()).astype(np.float64)


def close(got, ref, extra, what):
    bound = 2.0 ** -8 * np.abs(ref) + extra + 2.0 ** -134
    worst = float(np.max(np.abs(got - ref) / bound, initial=0.0))
    differ = int((got != bf16(ref)[0]).sum())
    print(f"  {what}: error / bound {worst:.3f}, {differ} of {ref.size} not correctly rounded", flush=True)
    assert worst <= 1.0 and differ <= 1 + ref.size // 100


SHAPES = [(1, 1), (1, 64), (3, 7), (2, 512), (5, 520), (4, 1015), (3, 1024), (2, 1032), (3, 2048), (2, 2056), (1, 4096),
          (1, 6144), (7, 6144), (2, 6152), (2, 8192), (2, 9999), (1, 16384),
          (2050, 1049), (2049, 1999)]  # the last two: one wave a row for many rows


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("pad", [0, 5, 8])
def test_norm_in(ops, T, H, pad):
    say(f"norm_in {T}x{H}+{pad}")
    rng = np.random.default_rng(H + T)
    x, xb = bf16(rng.standard_normal((T, H + pad)) * np.exp(rng.standard_normal((T, 1))))
    w, wb = bf16(1 + 0.3 * rng.standard_normal(H))
    out = torch.full((T, H + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_norm_in(dev_bf16(xb)[:, :H], dev_bf16(wb), EPS, n=out[:, :H])
    ref = onorm.norm(x[:, :H], w, EPS)
    close(values(out[:, :H]), ref, (H + 16) * U * np.abs(ref), "n")
    assert bool((out[:, H:] == 7.0).all())


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
def test_norm_out(ops, T, H, gate, y_dtype):
    say(f"norm_out {T}x{H} {gate} {y_dtype}")
    rng = np.random.default_rng(H + T + len(gate))
    y32 = (rng.standard_normal((T, H)) * 3).astype(np.float32)
    if y_dtype == torch.bfloat16:
        y, yb = bf16(y32)
        yd = dev_bf16(yb)
    else:
        y, yd = y32.astype(np.float64), torch.from_numpy(y32).cuda()
    r, rb = bf16(rng.standard_normal((T, H)))
    wp, wpb = bf16(1 + 0.3 * rng.standard_normal(H))
    wn, wnb = bf16(1 + 0.3 * rng.standard_normal(H))
    shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[gate]
    g, gd = None, None
    if shape is not None:
        g, gb = bf16(rng.standard_normal(shape))
        gd = dev_bf16(gb)
    rd, wpd, wnd = dev_bf16(rb), dev_bf16(wpb), dev_bf16(wnb)
    for post in (True, False):
        ref = onorm.residual(y, r, wp if post else None, g, 0.25, EPS)
        z = np.abs(ref - r)
        out, n = ops.moe_norm_out(yd, rd, wpd if post else None, wnd, gate=gd, residual_scale=0.25, eps=EPS)
        close(values(out), ref, (H + 16) * U * (z + np.abs(r)), "r'")
        n_ref = onorm.norm(values(out), wn, EPS)  # the next norm reads the residual that is kept
        close(values(n), n_ref, (H + 16) * U * np.abs(n_ref), "n")
    assert torch.equal(ops.moe_norm_out(yd, rd, wpd, gate=gd, residual_scale=0.25, eps=EPS),
                       ops.moe_norm_out(yd, rd, wpd, wnd, gate=gd, residual_scale=0.25, eps=EPS)[0])
    inplace = rd.clone()
    ops.moe_norm_out(yd, inplace, wpd, wnd, gate=gd, residual_scale=0.25, eps=EPS, out=inplace)
    assert torch.equal(inplace, ops.moe_norm_out(yd, rd, wpd, gate=gd, residual_scale=0.25, eps=EPS))


@pytest.mark.parametrize("T,H,pad", [(1, 32, 0), (3, 288, 8), (5, 992, 3), (2, 2048, 0), (3, 4128, 0), (4, 6144, 0),
                                     (2, 16384, 8)])
def test_quantized_norms(ops, T, H, pad):
    """The MXFP4 form equals mxfp4_quantize of the BF16 result, bit for bit, with and without that result."""
    rng = np.random.default_rng(H)
    x = dev_bf16(bf16(rng.standard_normal((T, H + pad)))[1])[:, :H]
    y = dev_bf16(bf16(rng.standard_normal((T, H + pad)))[1])[:, :H]
    w = dev_bf16(bf16(1 + 0.3 * rng.standard_normal(H))[1])
    n, codes, scales = ops.moe_norm_in(x, w, EPS, quantize=True)
    assert torch.equal(n, ops.moe_norm_in(x, w, EPS))
    c, s = ops.mxfp4_quantize(n)
    assert torch.equal(codes, c) and torch.equal(scales, s)
    none, c, s = ops.moe_norm_in(x, w, EPS, n=False, quantize=True)
    assert none is None and torch.equal(codes, c) and torch.equal(scales, s)
    out, n, codes, scales = ops.moe_norm_out(y, x, w, w, quantize=True)
    want = ops.moe_norm_out(y, x, w, w)
    assert torch.equal(out, want[0]) and torch.equal(n, want[1])
    c, s = ops.mxfp4_quantize(n)
    assert torch.equal(codes, c) and torch.equal(scales, s)


def test_norm_special_rows(ops):
    """A zero row stays zero, a row with a NaN is NaN and reaches no other, an infinity gives NaN where x is infinite."""
    H = 544
    x32 = np.random.default_rng(0).standard_normal((4, H)).astype(np.float32)
    x32[0] = 0
    x32[1, 9] = np.nan
    x32[2, 9] = np.inf
    x, xb = bf16(x32)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    n, codes, scales = ops.moe_norm_in(dev_bf16(xb), w, EPS, quantize=True)
    v = values(n)
    assert (v[0] == 0).all() and np.isnan(v[1]).all() and np.isnan(v[2, 9]) and (np.delete(v[2], 9) == 0).all()
    close(v[3:], onorm.norm(x[3:], np.ones(H), EPS), 1e-5 * np.abs(v[3:]), "n")
    assert (to_np(scales)[1, : H // 32] == 255).all() and to_np(scales)[2, 0] == 255
    c, s = ops.mxfp4_quantize(n)
    assert torch.equal(codes, c) and torch.equal(scales, s)
    out = ops.moe_norm_out(dev_bf16(xb), dev_bf16(xb), w)
    assert (values(out)[0] == 0).all() and np.isnan(values(out)[1]).all()


def test_norm_no_rows(ops):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert tuple(ops.moe_norm_in(e, w).shape) == (0, 64)
    out, n = ops.moe_norm_out(e, e, w, w)
    assert tuple(out.shape) == (0, 64) and tuple(n.shape) == (0, 64)
