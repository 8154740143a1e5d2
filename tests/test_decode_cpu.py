"""Refusals of the MXFP4 calls and the few-token layer: every one before the GPU is touched."""
import ctypes

import pytest

import bit_quantized_moe_token_b200 as moe
from bit_quantized_moe_token_b200._binding import _CLayer, _CLayerMX

OK, ARG, SHAPE, ALIGN, WS = 0, -1, -2, -3, -4
P = 1 << 20


def test_quant_rows():
    f = moe.lib().mxfp4_quant_rows
    assert f(P, 0, 0, 64, 64, P, P, None) == OK                # no rows
    assert f(P, 0, 4, 48, 48, P, P, None) == SHAPE
    assert f(P, 0, 4, 0, 0, P, P, None) == ARG
    assert f(P, 0, -1, 64, 64, P, P, None) == ARG
    assert f(P, 3, 4, 64, 64, P, P, None) == ARG               # unknown type
    assert f(P, 0, 4, 64, 63, P, P, None) == ARG               # rows that overlap
    assert f(P, 0, 4, 64, 68, P, P, None) == ALIGN             # 136-byte rows
    assert f(P + 2, 0, 4, 64, 64, P, P, None) == ALIGN
    assert f(P, 0, 4, 64, 64, P + 2, P, None) == ALIGN
    assert f(None, 0, 4, 64, 64, P, P, None) == ARG
    assert f(P, 0, 4, 64, 64, None, P, None) == ARG
    assert f(P, 0, 4, 64, 64, P, None, None) == ARG
    assert f(P, 0, 1 << 40, 64, 64, P, P, None) == SHAPE


def test_dequant_rows():
    f = moe.lib().mxfp4_dequant_rows
    assert f(P, P, 0, 64, P, 0, None) == OK
    assert f(P, P, 2, 40, P, 0, None) == SHAPE
    assert f(P, P, 2, 64, P, 1, None) == ARG                   # f16 would overflow
    assert f(P, P, 2, 64, P + 8, 0, None) == ALIGN
    assert f(P, None, 2, 64, P, 0, None) == ARG


def test_matmul():
    f = moe.lib().mxfp4_matmul
    assert f(P, P, P, P, 0, 8, 64, P, 0, None) == OK
    assert f(P, P, P, P, 8, 0, 64, P, 0, None) == OK
    assert f(P, P, P, P, 8, 8, 63, P, 0, None) == SHAPE
    assert f(P, P, P, P, 8, 8, 1 << 17, P, 0, None) == SHAPE
    assert f(P, P, P, P, 1 << 23, 8, 64, P, 0, None) == SHAPE
    assert f(P, P, P, P, -1, 8, 64, P, 0, None) == ARG
    assert f(P, P, P, P, 8, 8, 0, P, 0, None) == ARG
    assert f(P, P, P, P, 8, 8, 64, P, 1, None) == ARG
    assert f(P, None, P, P, 8, 8, 64, P, 0, None) == ARG
    assert f(P + 4, P, P, P, 8, 8, 64, P, 0, None) == ALIGN
    assert f(P, P + 1, P, P, 8, 8, 64, P, 0, None) == ALIGN
    assert f(P, P, P, P, 8, 8, 64, P + 4, 0, None) == ALIGN


def _layer(fmt, E=8, H=256, N=128, n_shared=0, Ns=0, ptr=P, shared=None):
    w = [ptr] * 6
    sh = [shared] * 3
    if fmt == "w4a8":
        return _CLayer(E, H, N, 128, *w, n_shared, Ns, *sh)
    return _CLayerMX(E, H, N, *w, n_shared, Ns, *sh)


@pytest.mark.parametrize("fmt", ["w4a8", "mxfp4"])
@pytest.mark.parametrize("tail", ["decode", "decode_router"])
def test_layer(fmt, tail):
    L = moe.lib()
    f, size = getattr(L, f"moe_{fmt}_{tail}"), getattr(L, f"moe_{fmt}_decode_workspace_bytes")
    r = ctypes.byref
    big = 1 << 40

    def call(layer, T=4, k=2, x=P, lg=P, out=P, ws=P, n=big):
        st = f(r(layer), x, lg, T, k, out, ws, n, None)
        if st in (SHAPE,) or T < 0 or k < 1:
            assert size(r(layer), T, k) == 0
        return st

    good = _layer(fmt)
    assert size(r(good), 4, 2) > 0
    assert call(good, T=0) == OK
    assert call(good, T=17) == SHAPE
    assert call(good, T=-1) == ARG
    assert call(good, k=0) == ARG
    assert call(good, k=9) in (ARG, SHAPE)
    assert call(_layer(fmt, E=0)) == ARG
    assert call(_layer(fmt, E=2000), k=2) in (ARG, SHAPE)
    assert call(_layer(fmt, H=200)) == SHAPE
    assert call(_layer(fmt, N=64)) == SHAPE
    assert call(_layer(fmt, H=16512)) == SHAPE
    assert call(_layer(fmt, N=8320)) == SHAPE
    assert call(_layer(fmt, H=8320), T=9) == SHAPE             # two blocks of eight tokens of more than 8192
    assert size(r(_layer(fmt, H=8320)), 8, 2) > 0
    assert call(_layer(fmt, n_shared=1, Ns=100, shared=P)) == SHAPE
    assert call(_layer(fmt, n_shared=1, Ns=8320, shared=P)) == SHAPE
    assert call(_layer(fmt, n_shared=-1)) == ARG
    assert call(_layer(fmt, n_shared=1, Ns=128)) == ARG        # shared experts without weights
    assert call(_layer(fmt, ptr=None)) == ARG
    assert call(_layer(fmt, ptr=P + 8)) == ALIGN
    assert call(good, x=None) == ARG
    assert call(good, lg=None) == ARG
    assert call(good, out=None) == ARG
    assert call(good, x=P + 2) == ALIGN
    assert call(good, out=P + 2) == ALIGN
    assert call(good, lg=P + 2) == ALIGN
    assert call(good, ws=None) == WS
    assert call(good, n=size(r(good), 4, 2) - 1) == WS
    assert call(good, ws=P + 64) == ALIGN
    assert f(None, P, P, 4, 2, P, P, big, None) == ARG
    if fmt == "w4a8":
        bad = _layer(fmt)
        bad.group = 64
        assert call(bad) == SHAPE


def test_names_are_public():
    for n in ("quant_mxfp4", "dequant_mxfp4", "matmul_mxfp4", "make_layer_mxfp4", "decode", "decode_router",
              "alloc_decode_workspace", "LayerMX", "mxfp4_quant_rows", "mxfp4_dequant_rows", "mxfp4_matmul",
              "moe_w4a8_decode", "moe_w4a8_decode_router", "moe_mxfp4_decode", "moe_mxfp4_decode_router"):
        assert n in moe.__all__ and hasattr(moe, n)
