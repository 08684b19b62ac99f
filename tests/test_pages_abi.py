"""The pages' and axes' C ABI on the host: struct layout and refusals (no GPU)."""
import ctypes
import os
import subprocess

import compressed_linear_amd as cla
from test_abi import ROOT
from test_serving_abi import ODD, P, cache


def pool(**kw):
    c = cla.cl_page_pool(256, 256, 512, 256, 3, 4, 8, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_struct_layout(tmp_path):
    prog = tmp_path / "sz.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "cl_int8.h"\n'
                    'int main(void){printf("%zu %zu\\n", sizeof(cl_page_pool), offsetof(cl_page_pool, page_size));return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(cla.cl_page_pool), cla.cl_page_pool.page_size.offset]


def test_pool_refuses():
    L = cla.lib()
    r = ctypes.byref
    calls = (lambda p: L.cl_pool_extend(p, P, 5, P, P, P, None), lambda p: L.cl_pool_fork(p, P, None),
             lambda p: L.cl_pool_truncate(p, ctypes.c_void_p(1024), None), lambda p: L.cl_pool_compact(p, 4, P, P, P, 1 << 30, None))
    for call in calls:
        assert call(None) == -1
        for kw in (dict(block_table=0), dict(lens=0), dict(refs=0), dict(left_out=0), dict(refs=258), dict(sequences=0), dict(width=0),
                   dict(pages=0), dict(page_size=0), dict(page_size=8), dict(page_size=24), dict(page_size=2048)):
            assert call(r(pool(**kw))) == -1, kw
            assert L.cl_last_error()
        for kw in (dict(sequences=4097), dict(pages=1 << 27), dict(width=1 << 27)):
            assert call(r(pool(**kw))) == -5, kw
    p = r(pool())
    for a in ((None, 5, P, P, P), (P, -1, P, P, P), (P, 5, None, P, P), (P, 5, P, None, P), (P, 5, P, P, ODD), (ODD, 5, P, P, P)):
        assert L.cl_pool_extend(p, *a, None) == -1, a
    assert L.cl_pool_fork(p, None, None) == -1 and L.cl_pool_fork(p, ODD, None) == -1
    assert L.cl_pool_truncate(p, None, None) == -1 and L.cl_pool_truncate(p, P, None) == -1  # the pool's own lens
    for a, st in (((-1, P, P, P, 99), -1), ((4, None, P, P, 99), -1), ((4, P, P, None, 99), -1), ((4, P, ODD, P, 99), -1),
                  ((4, P, P, P, 35), -3), ((0, None, None, None, 0), 0)):
        assert L.cl_pool_compact(p, *a, None) == st, a
    assert L.cl_pool_compact_work_bytes(8) == 36 and L.cl_pool_compact_work_bytes(0) == 0


def test_moves_refuse():
    L = cla.lib()
    r = ctypes.byref
    good = cache()
    for c, st in ((cache(k=0), -1), (cache(page_size=48), -1), (cache(dim=96), -2), (cache(kind=7), -1)):
        assert L.cl_kv_copy_pages(r(c), P, P, 3, None) == st
        assert L.cl_kv_keep(r(c), P, 2, 3, P, P, 4, None) == st
    for a, st in (((None, P, 3), -1), ((P, ODD, 3), -1), ((P, P, -1), -1), ((None, None, 0), 0)):
        assert L.cl_kv_copy_pages(r(good), *a, None) == st, a
    assert L.cl_kv_copy_pages(r(cache(k_scale=264)), P, P, 3, None) == -1
    for a, st in (((None, 2, 3, P, P, 4), -1), ((P, 0, 3, P, P, 4), -1), ((P, 2, -1, P, P, 4), -1), ((P, 2, 3, None, P, 4), -1),
                  ((P, 2, 3, P, ODD, 4), -1), ((P, 2, 3, P, P, -1), -1), ((P, 2, 3, P, P, 257), -2), ((P, 2, 70000, P, P, 4), -5),
                  ((None, 2, 0, None, None, 4), 0), ((None, 2, 3, None, None, 0), 0)):
        assert L.cl_kv_keep(r(good), *a, None) == st, a


def test_axes_refuse():
    L = cla.lib()

    def sections(*n):
        return (ctypes.c_int32 * len(n))(*n)

    def rope(s=sections(16, 8, 8), axes=3, order=0, tokens=3, pos=P, rot=64):
        return L.cl_rope_axes(P, 0, 128, 64, tokens, 2, 64, pos, axes, s, order, P, 8, rot, 0, ctypes.c_void_p(1024), 0, 128, 64, None)

    def append(s=sections(16, 8, 8), axes=3, order=0, tokens=3, pos=P, rot=64):
        return L.cl_kv_append_axes(ctypes.byref(cache()), P, P, 0, tokens, 128, 64, 128, 64, P, pos, axes, s, order, P, 8, rot, 0, None)

    for call in (rope, append):
        for kw in (dict(axes=0), dict(axes=5), dict(order=2), dict(order=-1), dict(axes=2), dict(s=sections(16, 8, 9)), dict(pos=None),
                   dict(s=sections(40, -8, 0)), dict(s=sections(4, 24, 4), order=1), dict(s=sections(2 ** 31 - 1, 2 ** 31 - 1, 34)),
                   dict(rot=62)):
            assert call(**kw) == -1, kw
            assert L.cl_last_error()
        assert call(tokens=0) == 0
