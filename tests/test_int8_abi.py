"""The 8-bit integer layer's C ABI on the host: exported symbols and refusals (no GPU)."""
import ctypes
import os

import pytest

import compressed_linear_amd as cla
from test_abi import ROOT, header_functions

P = ctypes.c_void_p(256)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(257)


def test_header_and_library_agree():
    assert set(header_functions(os.path.join(ROOT, "include", "cl_int8.h"))) == set(cla.INT8_SYMBOLS)
    assert all(hasattr(cla.lib(), n) for n in cla.INT8_SYMBOLS)


def test_quant_refuses():
    L = cla.lib()

    def call(x=P, dtype=0, rows=3, K=100, clamp=0.0, codes=P, row=128, scale=P):
        return L.cl_int8_quant(x, dtype, 100, rows, K, clamp, codes, row, scale, None)

    for kw in (dict(x=None), dict(x=ODD), dict(dtype=3), dict(rows=-1), dict(K=0), dict(clamp=-1.0), dict(clamp=float("inf")),
               dict(clamp=float("nan")), dict(codes=None), dict(codes=ctypes.c_void_p(264)), dict(row=100), dict(row=0),
               dict(K=129), dict(scale=None), dict(scale=ODD)):
        assert call(**kw) == -1, kw
        assert L.cl_last_error()
    assert call(K=131072, row=131072) == -5
    assert call(rows=0, x=None) == 0


def test_linear_refuses():
    L = cla.lib()

    def linear(codes=P, row=128, scale=P, tokens=3, w=P, w_row=128, ws=P, bias=None, N=4, K=100, y=P, yd=0, work=P, size=1 << 40):
        return L.cl_int8_linear(codes, row, scale, tokens, w, w_row, ws, bias, N, K, y, yd, 4, work, size, None)

    def forward(x=P, dtype=0, tokens=3, clamp=0.0, w=P, w_row=128, ws=P, bias=None, N=4, K=100, y=P, yd=0, work=P, size=1 << 40):
        return L.cl_int8_forward(x, dtype, 100, tokens, clamp, w, w_row, ws, bias, N, K, y, yd, 4, work, size, None)

    for call in (linear, forward):
        for kw in (dict(tokens=-1), dict(w=None), dict(w=ctypes.c_void_p(264)), dict(w_row=64), dict(w_row=130), dict(ws=None),
                   dict(bias=ODD), dict(N=0), dict(K=0), dict(K=129), dict(y=None), dict(y=ODD), dict(yd=3)):
            assert call(**kw) == -1, kw
            assert L.cl_last_error()
        assert call(K=131072, w_row=131072) == -5
        assert call(tokens=0, w=None) == 0
    for kw in (dict(codes=None), dict(row=64), dict(scale=None), dict(codes=ODD)):
        assert linear(**kw) == -1, kw
    for kw in (dict(x=None), dict(dtype=-1), dict(x=ODD), dict(clamp=-2.0)):
        assert forward(**kw) == -1, kw
    assert linear(row=(1 << 23) + 128) == -5 and linear(w_row=(1 << 23) + 128) == -5
    for bad in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (5, 5, 131072)):
        assert L.cl_int8_work_bytes(*bad, 0) == 0 and L.cl_int8_work_bytes(*bad, 1) == 0
    need = L.cl_int8_work_bytes(4096, 4, 100, 0)
    assert need >= 4096 * 132
    assert forward(tokens=4096, size=need - 1) == -3
    assert forward(tokens=4096, work=None) == -1 and forward(tokens=4096, work=ctypes.c_void_p(264)) == -1
    # few tokens of many channels: K is cut into parts
    need = L.cl_int8_work_bytes(200, 1000, 100000, 1)
    assert need >= 2 * 4 * 200 * 1000 and need < L.cl_int8_work_bytes(200, 1000, 100000, 0)
    assert linear(tokens=200, N=1000, K=100000, row=100096, w_row=100096, size=need - 1) == -3


@pytest.mark.parametrize("clamp", [1e-30, 1e-45, 1e-50, 5e-324])
def test_a_small_clamp_stays_one(clamp):
    """The entries take a clamp of 0 as none, so one that a float cannot hold must not become 0."""
    from compressed_linear_amd.int8 import _clamp
    assert ctypes.c_float(_clamp(clamp)).value > 0.0
