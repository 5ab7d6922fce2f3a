"""Pins of the MXFP4 and norm oracle: closed forms, brute force, invariants (CPU only)."""

import numpy as np
import pytest

from oracle import formats, mx
from oracle import norm as onorm


def test_scale_bytes_of_powers_of_two():
    for e in range(-149, 128):
        assert mx.scale_byte(np.float64(2.0) ** e) == max(e - 2 + 127, 0)
        assert mx.scale_byte(np.nextafter(np.float64(2.0) ** (e + 1), 0)) == max(e - 2 + 127, 0)
    assert mx.scale_byte(0.0) == 0 and mx.scale_byte(np.inf) == 255 and mx.scale_byte(np.nan) == 255
    assert mx.scale_value(np.array([0, 127, 254])).tolist() == [2.0 ** -127, 1.0, 2.0 ** 127]
    assert np.isnan(mx.scale_value(np.array([255]))).all()


@pytest.mark.parametrize("v,code", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (7.9, 7),
                                    (0.26, 1), (0.74, 1), (5.01, 7), (6.0, 7)])
def test_rounding_and_saturation(v, code):
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1], x[0, 2] = 4.0, v, -v  # amax in [4, 8): the scale is 1
    codes, byte = mx.quantize(x)
    assert byte[0, 0] == 127 and codes[0, 1] == code and codes[0, 2] == (code | 8)


def test_every_representable_block_is_a_fixed_point():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (50, 64)).astype(np.uint8)
    codes[:, ::32] = 7  # a 6 in each block fixes the scale
    byte = rng.integers(1, 250, (50, 2)).astype(np.uint8)
    v = mx.dequantize(codes, byte)
    c2, b2 = mx.quantize(v)
    assert np.array_equal(b2, byte) and np.array_equal(formats.E2M1_VALUES[c2], formats.E2M1_VALUES[codes])


def test_error_is_at_most_half_a_step():
    x = np.random.default_rng(2).standard_normal((40, 96))
    q = mx.rounded(x)
    s = np.repeat(mx.scale_value(mx.quantize(x)[1]), 32, axis=1)
    a = np.abs(x) / s
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a <= 6, 1.0, 2.0)))
    assert (np.abs(q - x) / s <= half).all()


def test_nan_blocks():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.nan, -np.inf
    codes, byte = mx.quantize(x)
    assert byte[0, 0] == 255 and byte[1, 1] == 255 and (codes[0, :32] == 0).all()
    assert byte[0, 1] != 255 and np.isnan(mx.dequantize(codes, byte)[0, :32]).all()


def test_pack_reads_back_through_the_lane_rule():
    rng = np.random.default_rng(3)
    codes, byte = rng.integers(0, 16, (45, 288)).astype(np.uint8), rng.integers(0, 255, (45, 9)).astype(np.uint8)
    pc, ps = mx.pack(codes, byte)
    assert pc.shape == (2, 2, 4, 64, 16) and ps.shape == (2, 2, 64, 4)
    full = np.zeros((64, 512), np.uint8)
    sc = np.zeros((64, 16), np.uint8)
    for lane in range(64):  # every lane and piece names one block; together they name all
        f, m = lane // 32, lane % 32
        row = 16 * ((m >> 2) & 1) + 4 * (m >> 3) + (m & 3)
        for s in range(4):
            for g in range(2):
                for c in range(2):
                    blk = 8 * c + 4 * f + s
                    full[32 * g + row, 32 * blk: 32 * blk + 32: 2] = pc[g, c, s, lane] & 15
                    full[32 * g + row, 32 * blk + 1: 32 * blk + 32: 2] = pc[g, c, s, lane] >> 4
                    sc[32 * g + row, blk] = ps[g, c, lane, s]
    assert np.array_equal(full[:45, :288], codes) and np.array_equal(sc[:45, :9], byte)
    assert not full[45:].any() and not full[:, 288:].any() and not sc[45:].any() and not sc[:, 9:].any()


def test_grid_reach_covers_perturbed_inputs():
    rng = np.random.default_rng(4)
    h = rng.standard_normal((30, 64))
    h[:, ::32] = 4.0  # an amax on a power of two: the scale byte itself is in doubt
    delta = np.full_like(h, 0.02)
    q, reach = mx.grid_reach(h, delta)
    for _ in range(50):
        other = mx.rounded(h + delta * rng.uniform(-1, 1, h.shape))
        assert (np.abs(other - q) <= reach + 1e-15).all()
    assert mx.grid_reach(h, 0 * delta)[1].max() == 0


def test_pair_exponent_bounds_the_row():
    rng = np.random.default_rng(5)
    I = 96
    h = mx.quantize(rng.standard_normal((8, I)) * 3)
    w2 = mx.quantize(rng.standard_normal((64, I)))
    w = rng.uniform(0.01, 3, 8).astype(np.float32)
    f = mx.dequantize(*h) @ mx.dequantize(*w2).T * w[:, None]
    E = mx.pair_exponent(w, h[1].max(1), w2[1].max(), I)
    assert (np.abs(f) < 2.0 ** (E[:, None] + 15)).all()


def test_norm_closed_forms():
    v = np.array([[3.0, -4.0]])
    assert np.allclose(onorm.norm(v, [1.0, 2.0], 0.0), [[3 / np.sqrt(12.5), -8 / np.sqrt(12.5)]], rtol=1e-15)
    assert np.array_equal(onorm.norm(np.zeros((1, 4)), np.ones(4), 1e-6), np.zeros((1, 4)))
    a, b = onorm.norm(v, [1, 1], 0.0), onorm.norm(-7 * v, [1, 1], 0.0)
    assert np.allclose(a, -b, rtol=1e-15)
    assert np.array_equal(onorm.residual(v, 2 * v, None, np.array([[0.5]]), 2.0, 0.0), 3 * v)
