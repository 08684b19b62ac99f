"""Sizes past what a launch of the serving operators holds are refused on the host (no GPU)."""
import ctypes

import compressed_linear_amd as cla


def test_rope_of_too_many_heads():
    L, P = cla.lib(), ctypes.c_void_p(256)  # never dereferenced
    assert L.cl_rope(P, 0, 16, 16, 1, 1 << 30, 16, P, P, 8, 16, 0, ctypes.c_void_p(1 << 40), 0, 16, 16, None) == -5
    assert b"heads" in L.cl_last_error()
