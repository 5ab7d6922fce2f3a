"""RMS norms around a block (oracle), in float64.

norm:  v / sqrt(mean(v^2) + eps) * w.
out:   r' = r + s * gate * norm(y, w_post), then norm(r', w_next) on the r' that is stored.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

from __future__ import annotations

import numpy as np


def norm(v: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    v = np.asarray(v, np.float64)
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def residual(y, r, w_post, gate, scale: float, eps: float) -> np.ndarray:
    z = np.asarray(y, np.float64) if w_post is None else norm(y, w_post, eps)
    if gate is not None:
        z = z * np.asarray(gate, np.float64)
    return np.asarray(r, np.float64) + scale * z
