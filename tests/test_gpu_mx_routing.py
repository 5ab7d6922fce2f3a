"""GPU parity of the MXFP4 experts under routings that moe_route does not write.

The checks and their bounds are test_gpu_mx.test_experts', with the routing replaced by one made here."""

import numpy as np
import pytest
import torch

import test_gpu_mx as mxt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def routed(ids, rng):
    """ids [T, k] -> what test_gpu_mx.routing returns"""
    T, k = ids.shape
    w = rng.uniform(0.05, 1.5, (T, k)).astype(np.float32)
    flat = ids.reshape(-1)
    counts = np.bincount(flat, minlength=int(flat.max()) + 1)
    return ids, w, counts, np.argsort(flat, kind="stable").astype(np.int32)


def with_ids(monkeypatch, make):
    """test_experts routes by make(rng, T, E, k) -> ids from here on."""

    def routing(rng, T, E, k, kind):
        ids, w, counts, order = routed(make(rng, T, E, k), rng)
        counts = np.concatenate([counts, np.zeros(E - counts.size, counts.dtype)])
        return ids, w, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), order

    monkeypatch.setattr(mxt, "routing", routing)


# T tokens no more than a tile of 64 (128) tokens holds, their pairs several times as many
@pytest.mark.parametrize("T,E,k,H,I", [(64, 3, 2, 288, 96), (33, 4, 4, 96, 64), (5, 8, 8, 256, 128),
                                       (120, 16, 16, 2848, 1440)])
def test_repeated_experts(ops, monkeypatch, T, E, k, H, I):
    """A token that names an expert more than once: an expert then has more pairs than there are tokens."""

    def make(rng, T, E, k):
        ids = rng.integers(0, E, (T, k))
        ids[: (2 * T + 2) // 3] = E - 1  # two thirds of the tokens name the last expert k times
        return ids

    with_ids(monkeypatch, make)
    mxt.test_experts(ops, T, E, k, H, I, "repeated")
