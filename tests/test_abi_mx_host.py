"""Host-only checks of the MXFP4 and norm entry points: every refusal comes before any HIP call
(fake, aligned addresses are never dereferenced on this path)."""

import ctypes

import pytest
import torch

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p(0x10000)
P2 = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10002)
BYTE = ctypes.c_void_p(0x10001)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from nvfp4_w4a4_mixture_amd import _lib

    return _lib.lib()


def refuses(call, **cases):
    """Each keyword names an argument's bad value(s) and the expected status."""
    for name, pairs in cases.items():
        for value, status in pairs:
            assert call(**{name: value}) == status, (name, value)


def test_quantize_refusals(L):
    def q(x=P, dt=0, rows=4, cols=64, ld=64, codes=P, scales=P):
        return L.mxfp4_quantize(x, dt, rows, cols, ld, codes, scales, None)

    def d(x=P, dt=0, rows=4, cols=64, ld=64, codes=P, scales=P):
        return L.mxfp4_dequantize(codes, scales, rows, cols, dt, x, ld, None)

    for call in (q, d):
        refuses(call, x=[(None, NULL), (ODD, ALIGN)], dt=[(2, SHAPE), (-1, SHAPE)], rows=[(-1, SHAPE), (BIG, SHAPE)],
                cols=[(0, SHAPE), (48, SHAPE), (-32, SHAPE)], ld=[(32, SHAPE), (68, ALIGN)],
                codes=[(None, NULL), (ctypes.c_void_p(0x10004), ALIGN)], scales=[(None, NULL)])
        assert call(rows=1 << 30, cols=256, ld=256) == SHAPE  # past one launch
        assert call(rows=0, x=None, codes=None, scales=None) == OK
        assert call(dt=1, ld=66) == ALIGN
    assert b"mxfp4_dequantize" in L.moe_last_error()


def test_weight_refusals(L):
    def q(batch=2, N=33, K=64, w=P, codes=P, scales=P, ms=P):
        return L.mxfp4_quantize_weights(w, batch, N, K, codes, scales, ms, None)

    refuses(q, batch=[(-1, SHAPE), (BIG, SHAPE)], N=[(0, SHAPE), (BIG, SHAPE)], K=[(0, SHAPE), (48, SHAPE), (BIG, SHAPE)],
            w=[(None, NULL), (ODD, ALIGN)], codes=[(None, NULL), (ODD, ALIGN)], scales=[(None, NULL)], ms=[(ODD, ALIGN)])
    assert q(batch=0, w=None, codes=None, scales=None, ms=None) == OK

    def p(batch=2, N=33, K=64, a=P, b=ctypes.c_void_p(0x30000), pa=P2, pb=ctypes.c_void_p(0x40000)):
        return L.mxfp4_pack_weights(a, b, batch, N, K, pa, pb, None, None)

    def u(batch=2, N=33, K=64, a=P, b=ctypes.c_void_p(0x30000), pa=P2, pb=ctypes.c_void_p(0x40000)):
        return L.mxfp4_unpack_weights(pa, pb, batch, N, K, a, b, None)

    for call in (p, u):
        refuses(call, batch=[(-1, SHAPE)], N=[(0, SHAPE)], K=[(31, SHAPE)], a=[(None, NULL), (ODD, ALIGN), (P2, SHAPE)],
                b=[(None, NULL), (ctypes.c_void_p(0x40000), SHAPE)], pa=[(None, NULL), (ODD, ALIGN)], pb=[(None, NULL)])


def test_linear_refusals(L):
    ws = L.mxfp4_linear_workspace_bytes(4, 64, 40)

    def lin(x=P, xs=P, T=4, K=64, w=P, s=P, N=40, dt=0, y=P, ldy=40, wsp=P2, wsb=1 << 30):
        return L.mxfp4_linear(x, xs, T, K, w, s, N, dt, y, ldy, wsp, wsb, None)

    refuses(lin, x=[(None, NULL), (ODD, ALIGN)], xs=[(None, NULL), (ODD, ALIGN)], T=[(-1, SHAPE), (2097121, SHAPE)],
            K=[(0, SHAPE), (40, SHAPE)], w=[(None, NULL), (ODD, ALIGN)], s=[(None, NULL), (ODD, ALIGN)],
            N=[(0, SHAPE), (41, SHAPE)], dt=[(2, SHAPE)], y=[(None, NULL), (BYTE, ALIGN)], ldy=[(39, SHAPE)])
    assert lin(dt=1, y=ODD) == ALIGN
    assert lin(T=0, x=None, xs=None, y=None) == OK
    assert lin(T=1 << 20, K=8192) == SHAPE  # 4 GiB of x codes
    assert lin(N=(1 << 27) + 1, ldy=1 << 28) == SHAPE and lin(T=1 << 20, N=1 << 21, ldy=1 << 21) == SHAPE
    assert lin(ldy=1 << 31) == SHAPE
    if ws:
        assert lin(wsp=None) == WORKSPACE and lin(wsb=ws - 1) == WORKSPACE and lin(wsp=ODD) == ALIGN


def test_ffn_refusals(L):
    need = L.mxfp4_ffn_workspace_bytes(4, 2, 8, 256, 128)
    assert need > 0 and L.mxfp4_ffn_workspace_bytes(8, 2, 8, 256, 128) > need
    assert L.mxfp4_ffn_workspace_bytes(-1, 2, 8, 256, 128) == 0

    def ffn(T=4, H=256, E=8, I=128, k=2, ws=P2, wsb=1 << 30, **ptr):
        a = dict(x=P, xs=P, c13=P, s13=P, c2=P, s2=P, m2=P, off=P, srt=P, tw=P, po=P, ps=P)
        a.update(ptr)
        return L.mxfp4_grouped_ffn(a["x"], a["xs"], T, H, a["c13"], a["s13"], a["c2"], a["s2"], a["m2"], E, I, k,
                                   a["off"], a["srt"], a["tw"], a["po"], a["ps"], ws, wsb, None)

    refuses(ffn, T=[(-1, SHAPE), (1 << 31, SHAPE), (1 << 30, SHAPE)], H=[(0, SHAPE), (48, SHAPE), (1 << 24, SHAPE)],
            E=[(0, SHAPE), (1, SHAPE), (257, SHAPE)], I=[(0, SHAPE), (16, SHAPE)], k=[(0, SHAPE), (9, SHAPE)],
            ws=[(None, WORKSPACE), (ODD, ALIGN)], wsb=[(need - 1, WORKSPACE)])
    for n in ("x", "xs", "c13", "s13", "c2", "s2", "m2", "off", "srt", "tw", "po", "ps"):
        assert ffn(**{n: None}) == NULL, n
        assert ffn(**{n: ODD}) == ALIGN, n
    assert ffn(T=0, x=None) == OK
    assert ffn(T=1 << 21, H=4096) == SHAPE  # 4 GiB of x codes
    assert ffn(T=1 << 21, I=4096, H=32) == SHAPE  # 4 GiB of h codes
    assert ffn(T=1 << 20, I=32, H=1 << 16) == SHAPE and ffn(T=1 << 18, I=32, H=1 << 18) == SHAPE  # too many tiles


def test_norm_refusals(L):
    def nin(x=P, T=4, H=64, ldx=64, w=P, eps=1e-6, n=P, ldn=64, c=P, s=P):
        return L.moe_norm_in(x, T, H, ldx, w, eps, n, ldn, c, s, None)

    def nout(x=P, dt=0, T=4, H=64, ldx=64, r=P, ldr=64, wp=P, g=P, grs=0, gcs=1, w=P, eps=1e-6, ro=P, ldro=64, n=P,
             ldn=64, c=P, s=P):
        return L.moe_norm_out(x, dt, T, H, ldx, r, ldr, wp, g, grs, gcs, 1.0, w, eps, ro, ldro, n, ldn, c, s, None)

    nan = float("nan")
    for call in (nin, nout):
        refuses(call, x=[(None, NULL), (BYTE, ALIGN)], T=[(-1, SHAPE), (1 << 24, SHAPE)],
                H=[(0, SHAPE), (16385, SHAPE), (40, SHAPE)], ldx=[(63, SHAPE), (1 << 31, SHAPE)], eps=[(-1.0, SHAPE), (nan, SHAPE)],
                n=[(BYTE, ALIGN)], ldn=[(63, SHAPE), (1 << 31, SHAPE)], c=[(None, NULL), (ODD, ALIGN)], s=[(None, NULL)], w=[(BYTE, ALIGN)])
        assert call(n=None, c=None, s=None) == NULL
        assert call(T=0) == OK
    assert nin(w=None) == NULL
    refuses(nout, dt=[(2, SHAPE)], r=[(None, NULL), (BYTE, ALIGN)], ldr=[(63, SHAPE), (1 << 31, SHAPE)], ldro=[(63, SHAPE)],
            ro=[(None, NULL)], grs=[(-1, SHAPE), (1 << 31, SHAPE)], gcs=[(2, SHAPE)], wp=[(BYTE, ALIGN)], g=[(BYTE, ALIGN)], w=[(None, NULL)])
    assert nout(dt=1, x=ODD) == ALIGN


def test_binding_refusals():
    from nvfp4_w4a4_mixture_amd import ops

    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: ops.mxfp4_quantize(x), lambda: ops.moe_norm_in(x, x[0]),
                 lambda: ops.moe_norm_out(x, x), lambda: ops.mxfp4_quantize_weights(x[None])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        ops.mxfp4_quantize(x.to(torch.float16))
    with pytest.raises(ValueError, match=r"\[G, KK"):
        ops.mxfp4_linear(x, x, x, x, 3)
