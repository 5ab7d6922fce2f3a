"""buffers.Buffers: what is kept, what is dropped (CPU tensors; streams and capture are stood in for)."""

import pytest
import torch

from nvfp4_w4a4_mixture_amd import buffers


@pytest.fixture
def gpu(monkeypatch):
    state = {"capturing": False, "stream": 0, "recorded": []}
    monkeypatch.setattr(buffers, "_capturing", lambda: state["capturing"])
    monkeypatch.setattr(buffers, "_current_stream", lambda device: state["stream"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["stream"])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state["recorded"].append((t.data_ptr(), s)),
                        raising=False)
    return state


def make(n):
    return lambda: dict(a=torch.empty(n, dtype=torch.uint8), b=(torch.empty(n // 4, dtype=torch.float32), None), c=1)


def test_least_recently_used_sets_go_first(gpu):
    b = buffers.Buffers("cpu", keep_bytes=1000)
    first = b.take(1, make(200))
    b.take(2, make(200))
    assert b.bytes == 800 and list(b) == [1, 2]
    assert b.take(1, make(200)) is first and list(b) == [2, 1]
    b.take(3, make(200))
    assert list(b) == [1, 3] and b.bytes == 800
    held = b[3]["a"].fill_(7)
    b.take(4, make(400))  # both older ones have to go
    assert list(b) == [4] and b.bytes == 800 and bool((held == 7).all())


def test_a_set_beyond_the_bound_is_used_and_dropped_later(gpu):
    b = buffers.Buffers("cpu", keep_bytes=100)
    assert b.take("large", make(400))["a"].numel() == 400 and "large" in b
    b.take("small", make(40))
    assert list(b) == ["small"] and b.bytes == 80


def test_captured_sets_stay(gpu):
    b = buffers.Buffers("cpu", keep_bytes=1000)
    kept = b.take(1, make(400))
    gpu["capturing"] = True
    assert b.take(1, make(400)) is kept and b.bytes == 0
    made = b.take(2, make(400))  # first used in a capture
    gpu["capturing"] = False
    for n in range(3, 8):
        b.take(n, make(400))
    assert b[1] is kept and b[2] is made and b.bytes == 800 and 7 in b and 6 not in b
    assert b.take(1, make(400)) is kept and b.bytes == 800
    assert not gpu["recorded"]


def test_other_streams_are_recorded(gpu):
    b = buffers.Buffers("cpu")
    s = b.take(1, make(64))
    gpu["stream"] = 5
    b.take(1, make(64))
    assert gpu["recorded"] == [(s["a"].data_ptr(), 5), (s["b"][0].data_ptr(), 5)]
    b.take(2, make(64))
    assert len(gpu["recorded"]) == 2
