"""MXFP4 quantization, packing and products (oracle), in float64.

The format is the public OCP Microscaling (MX) v1.0 definition: 32 consecutive
elements of a row are E2M1 and share one E8M0 scale, byte b = 2**(b - 127),
255 = NaN.  Quantization follows its conversion rule: the shared exponent is
floor(log2(amax)) less the exponent of the largest element value (6 = 1.5 *
2**2), elements are rounded to nearest, ties to even, and saturate.  A block
holding a NaN or an infinity is a NaN block.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

from __future__ import annotations

import numpy as np

from . import formats

BLOCK = 32
NAN_BYTE = 255


def scale_value(byte: np.ndarray) -> np.ndarray:
    b = np.asarray(byte, dtype=np.int64)
    return np.where(b == NAN_BYTE, np.nan, np.ldexp(1.0, np.minimum(b, 254) - 127))


def scale_byte(amax: np.ndarray) -> np.ndarray:
    """Scale byte of a block from its largest magnitude (float64; NaN and inf give 255)."""
    a = np.asarray(amax, dtype=np.float64)
    finite = np.isfinite(a) & (a > 0)
    _, e = np.frexp(np.where(finite, a, 1.0))  # a = m * 2**e, m in [0.5, 1): floor(log2 a) = e - 1
    b = np.clip(e.astype(np.int64) - 1 - 2 + 127, 0, 254)
    return np.where(finite, b, np.where(a == 0, 0, NAN_BYTE)).astype(np.uint8)


def _round_codes(v: np.ndarray) -> np.ndarray:
    """Nearest E2M1 code of each v (float64), ties to the even code, saturating; sign bit from v."""
    mags = formats.E2M1_VALUES[:8]
    mid = (mags[:-1] + mags[1:]) / 2
    a = np.abs(v)
    below, upto = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")  # they differ on a tie only
    pick = np.where(below % 2 == 0, below, upto)  # of two neighbours exactly one code is even
    return (pick | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def quantize(x: np.ndarray, byte: np.ndarray | None = None) -> tuple[np.ndarray, np.ndarray]:
    """x [rows, cols], cols % 32 == 0 -> codes [rows, cols] (one per element), bytes [rows, cols / 32].

    ``byte`` fixes the scale bytes instead of taking them from the blocks."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, BLOCK)
    if byte is None:
        with np.errstate(invalid="ignore"):
            byte = scale_byte(np.abs(b).max(-1))
    nan = byte == NAN_BYTE
    v = np.where(nan[..., None], 0.0, b) / np.where(nan, 1.0, scale_value(np.where(nan, 127, byte)))[..., None]
    codes = np.where(nan[..., None], 0, _round_codes(v)).astype(np.uint8)
    return codes.reshape(x.shape), byte


def dequantize(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    v = formats.E2M1_VALUES[codes].reshape(codes.shape[0], -1, BLOCK) * scale_value(byte)[..., None]
    return v.reshape(codes.shape)


def rounded(x: np.ndarray) -> np.ndarray:
    return dequantize(*quantize(x))


def padded(cols: int) -> int:
    return -(-cols // 256) * 256


def row_form(codes: np.ndarray, byte: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """The padded row form of activations: packed codes [rows, Cp/2], bytes [rows, Cp/32]."""
    rows, cols = codes.shape
    c = np.zeros((rows, padded(cols)), np.uint8)
    c[:, :cols] = codes
    s = np.zeros((rows, padded(cols) // BLOCK), np.uint8)
    s[:, : cols // BLOCK] = byte
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), s


def pack(codes: np.ndarray, byte: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Packed weights of one matrix, written element by element from the layout's address rule:
    row 32 g + 16 h + 4 q + j, block 8 c + 4 f + s -> lane 32 f + 8 q + 4 h + j, piece s of (g, c)."""
    n, k = codes.shape
    g, kk = -(-n // 32), padded(k) // 256
    pc = np.zeros((g, kk, 4, 64, 16), np.uint8)
    ps = np.zeros((g, kk, 64, 4), np.uint8)
    two = (codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(n, k // BLOCK, 16)
    for r in range(n):
        h, q, j = (r % 32) // 16, (r % 16) // 4, r % 4
        for blk in range(k // BLOCK):
            f, s = (blk % 8) // 4, blk % 4
            lane = 32 * f + 8 * q + 4 * h + j
            pc[r // 32, blk // 8, s, lane] = two[r, blk]
            ps[r // 32, blk // 8, lane, s] = byte[r, blk]
    return pc, ps


def silu(g: np.ndarray) -> np.ndarray:
    return g / (1.0 + np.exp(-g))


def grid_reach(h: np.ndarray, delta: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Quantization of h [rows, cols] known only to within delta >= 0 elementwise.

    Returns (value of the quantized h, bound on how far the quantization of any
    h' with |h' - h| <= delta can be from it).  Rounding is monotone for a fixed
    scale, and the scale byte is monotone in the block's amax, so the extremes
    over the two end points and the bytes of the two extreme amax bound it."""
    q = rounded(h)
    hb, db = np.abs(h).reshape(h.shape[0], -1, BLOCK), delta.reshape(h.shape[0], -1, BLOCK)
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
    lg = int(np.ceil(np.log2(36 * I)))
    low = np.maximum(e - 1, 0) - 126  # w 2**-E stays finite
    return np.minimum(np.maximum((e - 1) + 1 + lg + h_byte.astype(np.int64) + w2_byte.astype(np.int64) - 269, low), 113)
