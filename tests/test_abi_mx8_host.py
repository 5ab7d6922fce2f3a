"""Host-only checks of the MXFP8 entry points: every refusal comes before any HIP call (fake addresses)."""

import ctypes

import pytest
from test_abi_mx_host import ALIGN, BIG, BYTE, NULL, ODD, OK, P, P2, SHAPE, WORKSPACE, refuses

P4 = ctypes.c_void_p(0x10004)
MAX = (1 << 63) - 1


@pytest.fixture(scope="module")
def L():
    from nvfp4_w4a4_mixture_amd import _lib

    return _lib.lib()


def test_quantize_refusals(L):
    def q(x=P, dt=0, rows=4, cols=64, ld=64, codes=P, scales=P):
        return L.mxfp8_quantize(x, dt, rows, cols, ld, codes, scales, None)

    def d(x=P, dt=0, rows=4, cols=64, ld=64, codes=P, scales=P):
        return L.mxfp8_dequantize(codes, scales, rows, cols, dt, x, ld, None)

    for call in (q, d):
        refuses(call, x=[(None, NULL), (ODD, ALIGN)], dt=[(2, SHAPE), (-1, SHAPE)],
                rows=[(-1, SHAPE), (BIG, SHAPE), (MAX, SHAPE)], cols=[(0, SHAPE), (48, SHAPE), (-32, SHAPE)],
                ld=[(32, SHAPE), (68, ALIGN), (MAX, ALIGN)], codes=[(None, NULL), (P4, ALIGN)], scales=[(None, NULL)])
        assert call(rows=1 << 30, cols=256, ld=256) == SHAPE  # past one launch
        assert call(rows=0, x=None, codes=None, scales=None) == OK
    assert b"mxfp8_dequantize" in L.moe_last_error()


def test_linear_refusals(L):
    def lin(x=P, xs=P, T=4, K=64, w=P, s=P, N=40, bias=P, act=0, r=P, rdt=0, ldr=40, dt=0, y=P2, ldy=40):
        return L.mxfp8_linear(x, xs, T, K, w, s, N, bias, act, r, rdt, ldr, dt, y, ldy, None)

    refuses(lin, x=[(None, NULL), (ODD, ALIGN)], xs=[(None, NULL), (ODD, ALIGN)],
            T=[(-1, SHAPE), (2097121, SHAPE), (MAX, SHAPE)], K=[(0, SHAPE), (40, SHAPE)], w=[(None, NULL), (ODD, ALIGN)],
            s=[(None, NULL), (ODD, ALIGN)], N=[(0, SHAPE), (41, SHAPE)], bias=[(BYTE, ALIGN)], act=[(-1, SHAPE), (5, SHAPE)],
            r=[(BYTE, ALIGN)], rdt=[(2, SHAPE), (-1, SHAPE)], ldr=[(39, SHAPE), (1 << 31, SHAPE), (MAX, SHAPE)], dt=[(2, SHAPE)],
            y=[(None, NULL), (BYTE, ALIGN)], ldy=[(39, SHAPE), (MAX, SHAPE)])
    assert lin(dt=1, y=ODD) == ALIGN and lin(rdt=1, r=ODD) == ALIGN
    assert lin(r=P2, rdt=1) == SHAPE and lin(r=P2, ldr=48) == SHAPE  # in place: the same type and stride
    assert lin(T=0, x=None, xs=None, y=None) == OK
    assert lin(T=1 << 19, K=8192) == SHAPE  # 4 GiB of x codes
    assert lin(N=(1 << 27) + 1, ldy=1 << 28, ldr=1 << 28) == SHAPE
    assert lin(r=None, rdt=7, ldr=0, T=0) == OK  # what belongs to a residual is not looked at without one


def test_ffn_refusals(L):
    T, H, E, I, k = 4, 256, 8, 128, 2
    need = L.mxfp8_ffn_workspace_bytes(T, k, E, H, I)
    assert need == 8 * 256 + 256  # h codes and scales, padded
    for a in [(MAX, 8, 8, 256, 128), (4, MAX, 8, 256, 128), (4, 2, 8, 256, MAX), (-1, 2, 8, 256, 128)]:
        assert L.mxfp8_ffn_workspace_bytes(*a) == 0

    def ffn(xc=P, xs=P, T=T, H=H, c13=P, s13=P, c2=P, s2=P, ms=P, E=E, I=I, k=k, off=P, srt=P, tw=P, po=P, ps=P, ws=P,
            wb=need):
        return L.mxfp8_grouped_ffn(xc, xs, T, H, c13, s13, c2, s2, ms, E, I, k, off, srt, tw, po, ps, ws, wb, None)

    refuses(ffn, xc=[(None, NULL), (ODD, ALIGN)], xs=[(None, NULL), (ODD, ALIGN)], T=[(-1, SHAPE), (1 << 31, SHAPE)],
            H=[(0, SHAPE), (40, SHAPE), (1 << 24, SHAPE)], I=[(0, SHAPE), (40, SHAPE), (1 << 24, SHAPE)],
            E=[(1, SHAPE), (257, SHAPE)], k=[(0, SHAPE), (9, SHAPE)], c13=[(None, NULL), (ODD, ALIGN)],
            c2=[(None, NULL), (ODD, ALIGN)], s13=[(None, NULL), (ODD, ALIGN)], s2=[(None, NULL), (ODD, ALIGN)],
            ms=[(None, NULL), (ODD, ALIGN)], off=[(None, NULL)], srt=[(None, NULL)], tw=[(None, NULL)], po=[(None, NULL), (ODD, ALIGN)],
            ps=[(None, NULL), (ODD, ALIGN)], ws=[(None, WORKSPACE), (P4, ALIGN)], wb=[(need - 1, WORKSPACE)])
    assert ffn(T=1 << 24, wb=MAX) == SHAPE and ffn(T=0, xc=None, ws=None, wb=0) == OK
    assert b"mxfp8_grouped_ffn" in (ffn(H=40), L.moe_last_error())[1]


def test_layer_refusals(L):
    T, H, E, I, k = 5, 288, 8, 96, 2
    need = L.mxfp8_moe_layer_workspace_bytes(T, H, E, k, I)
    assert need > 0
    for a in [(33, H, E, k, I), (-1, H, E, k, I), (T, 40, E, k, I), (T, H, 257, k, I), (T, H, E, 9, I), (T, H, E, 0, I),
              (T, H, E, k, 1 << 24), (T, MAX - 31, E, k, I), (T, H, MAX, MAX, I)]:
        assert L.mxfp8_moe_layer_workspace_bytes(*a) == 0

    def lay(x=P, T=T, H=H, ldx=H, wr=P, b=P, E=E, k=k, rsf=2.5, c13=P, s13=P, c2=P, s2=P, I=I, dt=0, y=P, ids=P, tw=P,
            ws=P, wb=need):
        return L.mxfp8_moe_layer(x, T, H, ldx, wr, b, E, k, rsf, c13, s13, c2, s2, I, dt, y, ids, tw, ws, wb, None)

    refuses(lay, x=[(None, NULL), (BYTE, ALIGN)], T=[(-1, SHAPE), (33, SHAPE)], H=[(0, SHAPE), (40, SHAPE)],
            ldx=[(H - 1, SHAPE), (1 << 31, SHAPE)], wr=[(None, NULL), (BYTE, ALIGN)], b=[(None, NULL), (ODD, ALIGN)],
            E=[(1, SHAPE), (257, SHAPE)], k=[(0, SHAPE), (9, SHAPE)], rsf=[(0.0, SHAPE), (-1.0, SHAPE), (float("nan"), SHAPE)],
            c13=[(None, NULL), (ODD, ALIGN)], s13=[(None, NULL), (ODD, ALIGN)], c2=[(None, NULL), (ODD, ALIGN)],
            s2=[(None, NULL), (ODD, ALIGN)], I=[(0, SHAPE), (40, SHAPE)], dt=[(2, SHAPE)], y=[(None, NULL), (P4, ALIGN)],
            ids=[(None, NULL), (ODD, ALIGN)], tw=[(None, NULL), (ODD, ALIGN)], ws=[(None, WORKSPACE), (P4, ALIGN)],
            wb=[(need - 1, WORKSPACE)])
    assert lay(T=0, x=None, y=None, ws=None, wb=0) == OK


def test_norm_refusals(L):
    def nin(x=P, T=4, H=64, ldx=64, w=P, eps=1e-6, n=P, ldn=64, codes=P, scales=P):
        return L.moe_norm_in_mxfp8(x, T, H, ldx, w, eps, n, ldn, codes, scales, None)

    def nout(x=P, dt=0, T=4, H=64, ldx=64, r=P, ldr=64, wp=P, g=None, grs=0, gcs=0, w=P, eps=1e-6, ro=P, ldo=64, n=P, ldn=64,
             codes=P, scales=P):
        return L.moe_norm_out_mxfp8(x, dt, T, H, ldx, r, ldr, wp, g, grs, gcs, 1.0, w, eps, ro, ldo, n, ldn, codes, scales, None)

    for call in (nin, nout):
        refuses(call, x=[(None, NULL), (BYTE, ALIGN)], T=[(-1, SHAPE), (BIG, SHAPE)],
                H=[(0, SHAPE), (40, SHAPE), (16416, SHAPE)], ldx=[(63, SHAPE), (MAX, SHAPE)], w=[(None, NULL)],
                eps=[(-1.0, SHAPE)], ldn=[(63, SHAPE)], codes=[(None, NULL), (P4, ALIGN)], scales=[(None, NULL)])
        assert call(T=0, x=None, codes=None, scales=None) == OK
    refuses(nout, dt=[(2, SHAPE)], r=[(None, NULL)], ro=[(None, NULL)], ldr=[(63, SHAPE)], ldo=[(63, SHAPE)])
    assert nout(g=P, grs=-1) == SHAPE and nout(g=P, gcs=2) == SHAPE
    assert b"moe_norm_out_mxfp8" in L.moe_last_error()
