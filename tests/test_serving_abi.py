"""The serving operators' C ABI on the host: exported symbols, struct layout, refusals (no GPU)."""
import ctypes
import os
import subprocess

import compressed_linear_amd as cla
from test_abi import ROOT, header_functions

HEADER = os.path.join(ROOT, "include", "cl_serving.h")
P = ctypes.c_void_p(256)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(257)


def cache(**kw):
    c = cla.cl_kv_cache(256, 256, 256, 256, 4, 16, 2, 64, 0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_header_and_library_agree(tmp_path):
    assert set(header_functions(HEADER)) == set(cla.SERVING_SYMBOLS)
    assert all(hasattr(cla.lib(), n) for n in cla.SERVING_SYMBOLS)
    prog = tmp_path / "sz.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "cl_serving.h"\n'
                    'int main(void){printf("%zu %zu\\n", sizeof(cl_kv_cache), offsetof(cl_kv_cache, kind));return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(cla.cl_kv_cache), cla.cl_kv_cache.kind.offset]


def test_rope_refusals():
    L = cla.lib()

    def table(positions=8, rot=64, base=1e4, scaling=0, factor=1.0, trained=4096, fast=32.0, slow=1.0, out=P):
        return L.cl_rope_table(positions, rot, base, scaling, factor, trained, fast, slow, out, None)

    nan = float("nan")
    for kw in (dict(positions=0), dict(rot=7), dict(rot=0), dict(out=None), dict(out=ctypes.c_void_p(260)), dict(base=1.0),
               dict(base=nan), dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, factor=nan),
               dict(scaling=2, factor=2.0, rot=2), dict(scaling=3, trained=0), dict(scaling=3, fast=1.0),
               dict(scaling=3, slow=0.0)):
        assert table(**kw) == -1, kw
        assert L.cl_last_error()
    assert table(rot=2048) == -5

    def rope(x=P, xd=0, tokens=3, heads=2, dim=64, pos=P, tab=P, rows=8, rot=64, layout=0, y=ctypes.c_void_p(1024), yd=0,
             yt=128):
        return L.cl_rope(x, xd, 128, 64, tokens, heads, dim, pos, tab, rows, rot, layout, y, yd, yt, 64, None)

    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(tab=None), dict(x=ODD), dict(y=ODD), dict(xd=3), dict(yd=-1),
               dict(tokens=-1), dict(heads=0), dict(dim=1), dict(rows=0), dict(rot=0), dict(rot=33), dict(rot=66),
               dict(layout=2), dict(y=P, yd=1), dict(y=P, yt=256), dict(tab=ctypes.c_void_p(260))):
        assert rope(**kw) == -1, kw
    assert rope(dim=2000, rot=64) == -5
    assert rope(tokens=2 ** 31 - 1, heads=2 ** 20) == -5
    assert rope(tokens=0, x=None, y=None) == 0


def test_cache_refusals():
    L = cla.lib()

    def append(c, k=P, v=P, dtype=0, tokens=3, slots=P, pos=None, tab=None, rows=0, rot=0, layout=0):
        return L.cl_kv_append(ctypes.byref(c) if c else None, k, v, dtype, tokens, 128, 64, 128, 64, slots, pos, tab, rows,
                              rot, layout, None)

    for kw in (dict(k=0), dict(v=0), dict(k_scale=0), dict(v_scale=0), dict(k=264), dict(v_scale=260), dict(kind=2),
               dict(pages=0), dict(heads=0), dict(page_size=0), dict(page_size=8), dict(page_size=48), dict(page_size=2048)):
        assert append(cache(**kw)) == -1, kw
        assert L.cl_kv_read(ctypes.byref(cache(**kw)), P, 3, P, P, 0, None) == -1, kw
    assert append(None) == -1
    assert append(cache(dim=96)) == -2
    assert append(cache(pages=2 ** 30)) == -5
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(dtype=3), dict(tokens=-1), dict(k=ODD),
               dict(tab=P), dict(tab=P, pos=P, rows=4, rot=66), dict(tab=P, pos=P, rows=4, rot=64, layout=5)):
        assert append(cache(), **kw) == -1, kw
    assert append(cache(), tokens=0, k=None) == 0
    c = ctypes.byref(cache())
    assert L.cl_kv_read(c, None, 3, P, P, 0, None) == -1
    assert L.cl_kv_read(c, P, 3, None, P, 0, None) == -1
    assert L.cl_kv_read(c, P, 3, P, ctypes.c_void_p(264), 0, None) == -1
    assert L.cl_kv_read(c, P, -1, P, P, 0, None) == -1
    assert L.cl_kv_read(c, P, 3, P, P, 7, None) == -1
    assert L.cl_kv_read(c, None, 0, None, None, 0, None) == 0


def test_attention_refusals():
    L = cla.lib()

    def call(q=P, dtype=0, qt=256, qh=64, tokens=4, heads=4, c=None, bt=P, width=2, seqs=1, ctx=P, cu=P, max_q=4, max_ctx=9,
             mask=None, words=0, scale=1.0, o=P, work=P, size=1 << 40):
        return L.cl_tree_attention(q, dtype, qt, qh, tokens, heads, ctypes.byref(c or cache()), bt, width, seqs, ctx, cu,
                                   max_q, max_ctx, mask, words, scale, o, work, size, None)

    for kw in (dict(q=None), dict(o=None), dict(bt=None), dict(ctx=None), dict(cu=None), dict(dtype=2), dict(qt=252),
               dict(qh=4), dict(q=ctypes.c_void_p(264)), dict(tokens=-1), dict(heads=3), dict(heads=0), dict(seqs=-1),
               dict(max_q=-1), dict(max_ctx=-1), dict(width=0), dict(mask=P, words=0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(c=cache(page_size=20))):
        assert call(**kw) == -1, kw
        assert L.cl_last_error()
    assert call(max_q=257) == -2
    assert call(c=cache(dim=32)) == -2
    assert call(seqs=70000) == -5
    assert call(tokens=0, q=None) == 0 and call(seqs=0) == 0 and call(max_q=0) == 0


def test_logprobs_refusals():
    L = cla.lib()

    def call(x=P, dtype=0, rows=2, vocab=100, ids=P, given=1, logp=P, ent=P, k=4, ti=P, tl=P):
        return L.cl_token_logprobs(x, dtype, vocab, rows, vocab, ids, given, logp, ent, k, ti, tl, None)

    for kw in (dict(x=None), dict(ids=None), dict(logp=None), dict(ent=None), dict(ti=None), dict(tl=None), dict(x=ODD),
               dict(dtype=5), dict(rows=-1), dict(vocab=0), dict(given=-1), dict(k=-1), dict(vocab=3)):
        assert call(**kw) == -1, kw
        assert L.cl_last_error()
    assert call(k=33) == -2
    assert call(vocab=(1 << 24) + 1) == -5
    assert call(rows=0, x=None) == 0


def test_recording_refuses():
    assert cla.lib().cl_recording(None, None) == -1


def test_call_refuses():
    L = cla.lib()
    pack = lambda *a: b"".join(int(v).to_bytes(8, "little", signed=True) for v in a)  # noqa: E731
    assert L.cl_call(0, None) == -1 and L.cl_call(-1, pack(0)) == -1 and L.cl_call(5, pack(0)) == -1
    # cl_rope: no tokens; dim out of range; heads past 32 bits (which would be 2)
    ok = [256, 0, 128, 64, 0, 2, 64, 256, 256, 8, 64, 0, 1024, 0, 128, 64, 0]
    assert L.cl_call(0, pack(*ok)) == 0
    for at, value in ((6, 2000), (5, 2 ** 32 + 2), (4, -1)):
        bad = list(ok)
        bad[at] = value
        assert L.cl_call(0, pack(*bad)) == (-5 if value == 2000 else -1), at
        assert L.cl_last_error()
