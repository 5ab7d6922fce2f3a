"""A block fed with ever new token counts: bounded memory, unchanged results, graphs that stay valid."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx_block():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import mx_block as _m

    return _m


def rows(T, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + T)
    return torch.randn(T, 512, generator=g, device="cuda").to(torch.bfloat16)


def held(b):
    from nvfp4_w4a4_mixture_amd.buffers import _tensors

    return sum(t.numel() * t.element_size() for s in b._bufs.values() for t in _tensors(s))


def test_block_of_many_token_counts(mx_block):
    counts = list(range(1, 40)) + [300, 5, 200]
    plain, tight = mx_block.random_block(seed=1), mx_block.random_block(seed=1)
    tight._bufs.keep_bytes = 2 << 20
    first = None
    for T in counts:
        x = rows(T)
        a, b = plain(x, x), tight(x, x)
        assert torch.equal(a.residual, b.residual) and torch.equal(a.codes, b.codes) and torch.equal(a.y, b.y)
        first = first or (b.y, b.y.clone())
        size = held(tight)
        assert size <= tight._bufs.keep_bytes or list(tight._bufs) == [(T, 512)]
    assert torch.equal(*first)  # a result that the caller kept, of a set that is gone
    assert len(plain._bufs) == len(set(counts)) > len(tight._bufs)


def test_captured_block_among_many_token_counts(mx_block):
    blk = mx_block.random_block(seed=2)
    blk._bufs.keep_bytes = 1 << 20
    x = rows(24)
    want = blk(x, x).y.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = blk(x, x)
    y = out.y.data_ptr()
    del out
    for T in range(1, 30):
        other = blk(rows(T, 1), rows(T, 2)).y
        blk._bufs[(24, 512)]["y"].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert blk._bufs[(24, 512)]["y"].data_ptr() == y and torch.equal(blk._bufs[(24, 512)]["y"], want)
        assert bool(torch.isfinite(other).all())


def test_block_on_two_streams(mx_block):
    blk = mx_block.random_block(seed=3)
    blk._bufs.keep_bytes = 0  # every new token count drops the set before it
    want = {T: blk(rows(T), rows(T)).y.clone() for T in (40, 41, 42)}
    side = torch.cuda.Stream()
    x = {T: rows(T) for T in want}
    for _ in range(3):
        for T in want:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                got = blk(x[T], x[T]).y.clone()
            torch.cuda.current_stream().wait_stream(side)
            assert torch.equal(got, want[T])
            assert torch.equal(blk(x[T], x[T]).y, want[T])


def test_nvfp4_layer_of_many_token_counts(mx_block):
    from nvfp4_w4a4_mixture_amd import workload_io
    from workloads import by_name

    cfg, dev = by_name("tiny"), torch.device("cuda:0")
    plain, _ = workload_io.build_layer(cfg, dev)
    tight, _ = workload_io.build_layer(cfg, dev)
    tight._bufs.keep_bytes = 1 << 20
    x = workload_io.tokens(cfg, dev)
    for T in list(range(1, 65)) + [64, 3]:
        for reap in (False, True):
            a, b = plain(x[:T], reap=reap), tight(x[:T], reap=reap)
            assert torch.equal(a.y, b.y) and (not reap or torch.equal(a.saliency, b.saliency))
            assert held(tight) <= tight._bufs.keep_bytes
    assert len(plain._bufs) == 128 > len(tight._bufs)
