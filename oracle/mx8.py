"""MXFP8 (E4M3) quantization and its reach (oracle), in float64.

The OCP Microscaling v1.0 rule as in ``mx``, for E4M3 elements: the shared
exponent is floor(log2(amax)) less that of the largest element (448 = 1.75 *
2**8), elements are rounded to nearest, ties to even, and saturate.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

from __future__ import annotations

import numpy as np

from . import formats, mx

_MAGS = formats.E4M3_VALUES[:127]  # 0 .. 448
_MID = (_MAGS[:-1] + _MAGS[1:]) / 2


def scale_byte(amax: np.ndarray) -> np.ndarray:
    a = np.asarray(amax, dtype=np.float64)
    finite = np.isfinite(a) & (a > 0)
    _, e = np.frexp(np.where(finite, a, 1.0))
    b = np.clip(e.astype(np.int64) - 1 - 8 + 127, 0, 254)
    return np.where(finite, b, np.where(a == 0, 0, mx.NAN_BYTE)).astype(np.uint8)


def _round_bytes(v: np.ndarray) -> np.ndarray:
    a = np.abs(v)
    below, upto = np.searchsorted(_MID, a, "left"), np.searchsorted(_MID, a, "right")  # they differ on a tie only
    pick = np.where(below % 2 == 0, below, upto)
    return (pick | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def quantize(x: np.ndarray, byte: np.ndarray | None = None) -> tuple[np.ndarray, np.ndarray]:
    """x [rows, cols], cols % 32 == 0 -> E4M3 bytes [rows, cols], scale bytes [rows, cols / 32]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, mx.BLOCK)
    if byte is None:
        with np.errstate(invalid="ignore"):
            byte = scale_byte(np.abs(b).max(-1))
    nan = byte == mx.NAN_BYTE
    v = np.where(nan[..., None], 0.0, b) / np.where(nan, 1.0, mx.scale_value(np.where(nan, 127, byte)))[..., None]
    codes = np.where(nan[..., None], 0, _round_bytes(v)).astype(np.uint8)
    return codes.reshape(x.shape), byte


def dequantize(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    v = formats.E4M3_VALUES[codes].reshape(codes.shape[0], -1, mx.BLOCK) * mx.scale_value(byte)[..., None]
    return v.reshape(codes.shape)


def rounded(x: np.ndarray) -> np.ndarray:
    return dequantize(*quantize(x))


def row_form(codes: np.ndarray, byte: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """The padded row form of activations: bytes [rows, Cp], scales [rows, Cp/32]."""
    rows, cols = codes.shape
    c = np.zeros((rows, mx.padded(cols)), np.uint8)
    c[:, :cols] = codes
    s = np.zeros((rows, mx.padded(cols) // mx.BLOCK), np.uint8)
    s[:, : cols // mx.BLOCK] = byte
    return c, s


def grid_reach(h: np.ndarray, delta: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """As ``mx.grid_reach``: the value of the quantized h, and how far that of any h' within delta can be from it."""
    q = rounded(h)
    hb, db = np.abs(h).reshape(h.shape[0], -1, mx.BLOCK), delta.reshape(h.shape[0], -1, mx.BLOCK)
    top = scale_byte((hb + db).max(-1))
    low = scale_byte(np.maximum(hb - db, 0.0).max(-1))
    reach = np.zeros_like(h)
    for byte in (low, top):
        for end in (h - delta, h + delta):
            reach = np.maximum(reach, np.abs(dequantize(*quantize(end, byte)) - q))
    return q, reach


def pair_exponent(w: np.ndarray, h_byte: np.ndarray, w2_byte: np.ndarray, I: int) -> np.ndarray:
    """Exponent E of a pair row's scale 2**E (the header's rule); h_byte the row's largest, w2_byte the expert's."""
    _, e = np.frexp(np.asarray(w, np.float32))
    lg = int(np.ceil(np.log2(2688 * I)))
    low = np.maximum(e - 1, 0) - 126
    return np.minimum(np.maximum((e - 1) + 1 + lg + h_byte.astype(np.int64) + w2_byte.astype(np.int64) - 269, low), 113)
