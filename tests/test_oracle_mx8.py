"""Pins of the MXFP8 oracle: hand-worked blocks, ties, saturation, and the definition element by element."""

import numpy as np

from oracle import formats, mx, mx8


def block(*v):
    x = np.zeros((1, 32))
    x[0, : len(v)] = v
    return x


def test_hand_worked_blocks():
    # amax 448: scale 1; 1.0625 is a tie between 1.0 and 1.125 (even mantissa: 1.0); 1.1875 between 1.125 and 1.25 (1.25)
    codes, byte = mx8.quantize(block(448.0, 1.0625, 1.1875, -2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10))
    assert byte[0, 0] == 127
    assert list(mx8.dequantize(codes, byte)[0, :6]) == [448.0, 1.0, 1.25, -2.0 ** -9, 0.0, 2.0 ** -8]
    # amax just under a power of two saturates: 511 / 1 -> 448
    assert mx8.rounded(block(511.0))[0, 0] == 448.0
    assert mx8.rounded(block(512.0))[0, 0] == 512.0
    assert mx8.quantize(block(0.0))[1][0, 0] == 0 and mx8.quantize(block(-0.0))[0][0, 0] == 0x80
    for bad in (np.nan, np.inf, -np.inf):
        codes, byte = mx8.quantize(block(bad, 1.0))
        assert byte[0, 0] == 255 and not codes.any() and np.isnan(mx8.dequantize(codes, byte)).all()


def test_every_element_is_its_own_rounding():
    finite = [c for c in range(256) if c & 0x7F != 0x7F]
    v = formats.E4M3_VALUES[finite]
    assert np.array_equal(mx8._round_bytes(v), np.array(finite, np.uint8))
    gaps = np.diff(np.sort(np.unique(np.abs(v))))
    assert gaps.min() == 2.0 ** -9 and gaps.max() == 32.0


def test_rounding_is_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 64)) * np.exp2(rng.integers(-140, 100, (200, 1)))
    q = mx8.rounded(x)
    _, byte = mx8.quantize(x)
    unit = np.repeat(mx.scale_value(byte), 32, axis=1)
    a = np.minimum(np.abs(x) / unit, 448.0)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -6))), -6) - 3)
    assert (np.abs(np.abs(q) / unit - a) <= step / 2).all()
    assert (np.abs(q).reshape(200, 2, 32).max(-1) >= 0.875 * np.abs(x).reshape(200, 2, 32).max(-1)).all()


def test_row_form_pads_with_zeros():
    codes, byte = mx8.quantize(np.ones((2, 96)))
    c, s = mx8.row_form(codes, byte)
    assert c.shape == (2, 256) and s.shape == (2, 8) and not c[:, 96:].any() and not s[:, 3:].any()


def test_reach_covers_every_neighbour():
    rng = np.random.default_rng(2)
    h, d = rng.standard_normal((30, 64)), np.abs(rng.standard_normal((30, 64))) * 0.02
    q, reach = mx8.grid_reach(h, d)
    for _ in range(50):
        assert (np.abs(mx8.rounded(h + d * rng.uniform(-1, 1, h.shape)) - q) <= reach).all()
