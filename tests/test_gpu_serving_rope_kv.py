"""Rotary positions and the quantised K/V cache against plain references (needs an MI355X).

Rotation and quantisation are defined down to each fp32 rounding, so the kernels' bits are compared with
a plain fp32 evaluation; the definitions themselves are held against 64 bits.
"""
import sys

import numpy as np
import pytest

import compressed_linear_amd as cla
import serving_ref as ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dev_tensor(a, dtype="f32"):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(ref.torch_dtype(torch, dtype))


def ints(a):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def bits(t):
    torch = torch_cuda()
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16).cpu().numpy()


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 4.0), ("yarn", 8.0), ("yarn", 1.0)])
@pytest.mark.parametrize("P,rot", [(1, 2), (517, 64), (9000, 128), (70, 6)])
def test_table(scaling, factor, P, rot):
    if scaling == "ntk" and rot < 4:
        pytest.skip("the changed base needs two pairs")
    say("table", scaling, P, rot)
    got = cla.rope_table(P, rot, base=10000.0, scaling=scaling, factor=factor, trained=2048).cpu().numpy()
    want = ref.rope_table(P, rot, 10000.0, scaling, factor, 2048)
    # one rounding to fp32, and a few fp64 roundings of an angle of up to P
    assert (np.abs(got - want) <= 2.0 ** -24 * np.maximum(np.abs(want), 1e-30) * 1.001 + 64 * P * 2.0 ** -52).all()


def test_table_yarn_ends():
    # pairs that turn often keep their frequency, pairs that turn rarely are interpolated
    t = cla.rope_table(3, 128, scaling="yarn", factor=4.0, trained=4096).cpu().numpy().astype(np.float64)
    m = 0.1 * np.log(4.0) + 1.0
    assert abs(t[1, 0, 1] - m * np.sin(1.0)) < 1e-6
    w = 10000.0 ** (-126 / 128) / 4.0
    assert abs(t[2, 63, 1] - m * np.sin(2 * w)) < 1e-9


ROPE = [  # T, H, D, rot, layout, in, out
    (1, 72, 128, 128, "half", "f32", "bf16"), (7, 3, 128, 64, "interleaved", "bf16", "bf16"),
    (5, 2, 64, 64, "half", "f16", "f16"), (33, 5, 128, 32, "half", "f32", "f16"),
    (3, 1, 80, 20, "half", "f32", "f32"), (4, 2, 6, 2, "interleaved", "f16", "f32"),
    (2, 3, 7, 6, "half", "bf16", "f32"), (9, 2, 256, 256, "interleaved", "f32", "f32"),
    (130, 9, 96, 96, "half", "bf16", "f16"), (2, 2, 1024, 512, "half", "f16", "bf16"),
    (65, 4, 72, 40, "interleaved", "bf16", "f32"), (300, 80, 128, 128, "half", "f32", "bf16"),
    (45000, 3, 64, 32, "half", "bf16", "f16"), (18800, 7, 128, 128, "interleaved", "f16", "f32"),  # many tokens, odd heads
]


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("view", ["dense", "heads", "odd"])
def test_rope(case, view):
    T, H, D, rot, layout, src, dst = case
    torch = torch_cuda()
    r = np.random.default_rng(T * 1000 + D + rot)
    P = T + 40
    say("rope", case, view)
    whole = dev_tensor(r.normal(0, 2, (T, H + 3, D + 5)), src)
    if view == "dense":
        x = whole[:, :H, :D].contiguous()
    elif view == "heads":  # a view of a wider qkv buffer
        x = whole[:, :, :D].contiguous()[:, 2:2 + H]
    else:  # strides and a start that no vector divides
        x = whole[:, 1:1 + H, 3:3 + D]
    pos = r.integers(0, P, T)
    tab = ref.rope_table(P, rot).astype(np.float32)
    xf = x.float().cpu().numpy()
    want = torch.from_numpy(ref.rotate(xf, pos, tab, layout)).to(ref.torch_dtype(torch, dst))
    table = torch.from_numpy(tab).cuda()
    got = cla.rope(x, ints(pos), table, layout=layout, out_dtype=ref.torch_dtype(torch, dst))
    assert got.shape == x.shape and np.array_equal(bits(got), bits(want))
    exact = ref.rotate(xf.astype(np.float64), pos, tab, layout)
    err = np.abs(got.double().cpu().numpy() - exact)
    # two products and a sum in fp32 (of at most twice the largest input), then one rounding
    assert (err <= ref.U[dst] * np.abs(exact) * 1.001 + 4 * 2.0 ** -24 * 2 * np.abs(xf).max()).all()
    # into a given view of another buffer, and in place
    room = torch.full((T, H + 2, D + 3), 7.0, dtype=got.dtype, device="cuda")
    out = room[:, 1:1 + H, 2:2 + D]
    assert cla.rope(x, ints(pos), table, layout=layout, out=out) is out
    assert np.array_equal(bits(out), bits(want))
    room[:, 1:1 + H, 2:2 + D] = 7.0
    assert (room == 7.0).all()
    if src == dst:
        cla.rope(x, ints(pos), table, layout=layout, out=x)
        assert np.array_equal(bits(x), bits(want))


def test_rope_position_outside_the_table():
    torch = torch_cuda()
    x = dev_tensor(np.ones((4, 2, 64)))
    table = cla.rope_table(10, 32)
    y = cla.rope(x, ints([0, 10, -1, 9]), table).cpu().numpy()
    assert np.isnan(y[1:3, :, :32]).all() and (y[1:3, :, 32:] == 1).all()
    assert np.isfinite(y[[0, 3]]).all()
    assert cla.rope(x[:0], ints([]), table).shape == (0, 2, 64)
    torch.cuda.synchronize()


APPEND = [  # T, heads, D, page, kind, in, rot, layout
    (1, 8, 128, 64, "int8", "f32", 128, "half"), (1, 8, 128, 16, "int4", "bf16", 0, "half"),
    (37, 5, 128, 32, "int8", "bf16", 64, "interleaved"), (37, 5, 64, 16, "int4", "f32", 64, "half"),
    (300, 2, 128, 128, "int4", "f16", 128, "interleaved"), (129, 3, 64, 256, "int8", "f16", 32, "half"),
    (64, 1, 64, 1024, "int8", "f32", 20, "half"), (50, 8, 128, 16, "int4", "f32", 100, "half"),
    (1000, 8, 128, 64, "int8", "bf16", 128, "half"),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
@pytest.mark.parametrize("odd", [False, True])
def test_append_and_read(case, odd):
    T, H, D, page, kind, src, rot, layout = case
    torch = torch_cuda()
    r = np.random.default_rng(T + D + page + odd)
    say("append", case, odd)
    pages = -(-T // page) + 3
    lead = 3 if odd else 0
    qkv = dev_tensor(r.normal(0, 1, (T, 2 * H + 4, D + lead)) * np.exp(r.normal(0, 2, (T, 2 * H + 4, 1))), src)
    qkv[0, :, lead:] = 0  # a head of zeros
    k, v = qkv[:, 1:1 + H, lead:], qkv[:, 4 + H:4 + 2 * H, lead:]
    v[-1, 0, 1], v[-1, 0, 2] = float("nan"), float("inf")
    if D == 128 and T > 2:
        v[1, 0, 64:] = float("nan")
    cache = cla.KVCache(pages, page, H, D, kind)
    for t in (cache.k, cache.v):
        t.fill_(0xAB)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(float("nan"))
    slots = r.permutation(pages * page)[:T]
    skip = r.random(T) < 0.1
    skip[0] = False
    slots = np.where(skip, r.choice([-1, pages * page, -7], T), slots)
    pos, table, tab = None, None, None
    kf, vf = k.float().cpu().numpy(), v.float().cpu().numpy()
    if rot:
        P = 500
        tab = ref.rope_table(P, rot).astype(np.float32)
        pos = r.integers(0, P, T)
        table = torch.from_numpy(tab).cuda()
        kf = ref.rotate(kf, pos, tab, layout)
        if T > 3:
            pos[3] = P  # outside: stored as zeros
            kf[3] = 0
    cache.append(k, v, ints(slots), None if pos is None else ints(pos), table, layout)
    keep = np.flatnonzero(~skip)
    p, o = slots[keep] // page, slots[keep] % page
    for got_b, got_s, val in ((cache.k, cache.k_scale, kf), (cache.v, cache.v_scale, vf)):
        q, s = ref.quantise(val[keep], kind)
        gb, gs = got_b.cpu().numpy(), got_s.cpu().numpy()
        assert np.array_equal(gb[p, :, o], ref.codes_to_bytes(q, kind))
        assert np.array_equal(gs[p, :, o].view(np.uint16), s.view(np.uint16))
        if kind == "int4":  # at most 8 significant bits: code * scale is an fp16 value
            x = ref.stored(q, s, kind)
            big = np.abs(x) >= 2.0 ** -14
            assert (x[big].astype(np.float16).astype(np.float64) == x[big]).all()
        other = np.ones((pages, page), bool)
        other[p, o] = False
        assert (gb.transpose(0, 2, 1, 3)[other] == 0xAB).all()  # nothing else was touched
        assert np.isnan(gs.swapaxes(1, 2)[other].astype(np.float32)).all()
        # the definition against the values: half a step, or the clip that rounding the scale leaves
        fine = np.isfinite(val[keep])
        step = s.astype(np.float64)[..., None] if kind == "int8" else np.repeat(s.astype(np.float64), 32, -1)
        gap = np.abs(ref.stored(q, s, kind) - np.where(fine, val[keep], 0))
        clip = 127 * 2.0 ** -10 if kind == "int8" else 7 * 2.0 ** -8
        assert (gap <= step * (0.5 + clip) + 127 * 2.0 ** -25)[fine].all()
    ask = np.concatenate([slots[keep], [-1, pages * page]])
    for dst in ("f16", "bf16", "f32"):
        ko, vo = cache.read(ints(ask), dtype=ref.torch_dtype(torch, dst))
        for got, val in ((ko, kf), (vo, vf)):
            q, s = ref.quantise(val[keep], kind)
            x = torch.from_numpy(ref.stored(q, s, kind).astype(np.float32)).to(got.dtype)
            assert (got[:len(keep)].cpu() == x).all()  # exact: code * scale has at most 18 bits
            assert (got[len(keep):] == 0).all()


def test_append_nothing_and_last_slot():
    cache = cla.KVCache(2, 16, 1, 64, "int8")
    x = dev_tensor(np.ones((1, 1, 64)))
    cache.append(x[:0], x[:0], ints([]))
    cache.append(x, x, ints([31]))
    k, v = cache.read(ints([30, 31]))
    assert (k[0] == 0).all() and abs(float(k[1, 0, 0]) - 1.0) <= 2.0 ** -11
    assert cache.read(ints([]))[0].shape == (0, 1, 64)


def test_slots_past_4_gib():
    # codes past 2^32 bytes: 2^20 + 64 pages of 64 slots of 64 channels
    torch = torch_cuda()
    pages, page = (1 << 20) + 64, 64
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    cache = cla.KVCache(pages, page, 1, 64, "int8")
    r = np.random.default_rng(5)
    x = r.normal(0, 1, (3, 1, 64)).astype(np.float32)
    slots = [pages * page - 1, 5, (1 << 26) + 3]  # byte offsets 64 slot: 2^32 + 192, 320, the end
    t = dev_tensor(x)
    say("long cache append")
    cache.append(t, -t, ints(slots))
    q, s = ref.quantise(x, "int8")
    k, v = cache.read(ints(slots), dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy(), ref.stored(q, s, "int8").astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), -ref.stored(q, s, "int8").astype(np.float32))
    assert int((cache.k_scale != 0).sum()) == 3


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_other_stream_and_graph(kind):
    torch = torch_cuda()
    r = np.random.default_rng(77)
    T, H, D = 37, 4, 128
    table = cla.rope_table(200, D)
    k, v = (dev_tensor(r.normal(0, 1, (T, H, D)), "bf16") for _ in range(2))
    pos, slots = ints(r.integers(0, 200, T)), ints(r.permutation(64)[:T])

    def step(cache, k, v):
        q = cla.rope(k, pos, table, out_dtype=torch.float16)
        cache.append(k, v, slots, pos, table)
        return (q,) + cache.read(slots)

    caches = [cla.KVCache(2, 32, H, D, kind) for _ in range(3)]
    want = step(caches[0], k, v)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step(caches[1], k, v)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ki, vi = k.clone(), v.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step(caches[2], ki, vi)
    for i in range(4):
        ki.copy_(k * (1.0 + i))
        vi.copy_(v - i)
        want = step(caches[0], ki, vi)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_refusals():
    torch = torch_cuda()
    x = dev_tensor(np.ones((2, 3, 64)))
    table = cla.rope_table(8, 64)
    pos = ints([0, 1])
    for bad in (lambda: cla.rope(x.double(), pos, table), lambda: cla.rope(x[0], pos, table),
                lambda: cla.rope(x, pos.long(), table), lambda: cla.rope(x, ints([0]), table),
                lambda: cla.rope(x, pos, table[0]), lambda: cla.rope(x, pos, table.half()),
                lambda: cla.rope(x, pos, table, out=x[:, :2]), lambda: cla.rope(x, pos.cpu(), table),
                lambda: cla.rope(x, pos, table, out_dtype=torch.float64), lambda: cla.rope_table(0, 64),
                lambda: cla.rope_table(8, 5), lambda: cla.rope_table(8, 4, scaling="other"),
                lambda: cla.KVCache(1, 16, 1, 64, "int2"),
                lambda: cla.KVCache(k=torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(KeyError):
        cla.rope(x, pos, table, layout="other")
    with pytest.raises(cla.ClError):
        cla.rope(x[..., :32], pos, table)  # rot above dim
    with pytest.raises(cla.ClError):
        cla.rope(x, pos, table, out=x.view(torch.int16)[..., :64].view(torch.float16))  # y = x in another type
    cache = cla.KVCache(2, 16, 3, 64)
    s2 = ints([0, 1])
    for bad in (lambda: cache.append(x, x.half(), s2), lambda: cache.append(x[:, :2], x[:, :2], s2),
                lambda: cache.append(x, x, s2.long()), lambda: cache.append(x, x, s2, table=table),
                lambda: cache.append(x, x, ints([0])), lambda: cache.read(s2, dtype=torch.float64),
                lambda: cache.read(s2.long())):
        with pytest.raises(ValueError):
            bad()
    for sizes in ((2, 24, 1, 64), (2, 8, 1, 64), (2, 2048, 1, 64), (2, 16, 1, 96)):
        odd = cla.KVCache(*sizes)
        y = dev_tensor(np.ones((2, 1, sizes[3])))
        with pytest.raises(cla.ClError):
            odd.append(y, y, s2)
    torch.cuda.synchronize()
