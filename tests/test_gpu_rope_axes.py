"""Rotary positions with several axes against plain references (needs an MI355X), bit by bit in fp32 and against 64 bits."""
import sys

import numpy as np
import pytest

import compressed_linear_amd as cla
import serving_ref as ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def ints(a):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def bits(t):
    torch = torch_cuda()
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16).cpu().numpy()


def axis_of(sections, order):
    """Each pair's axis, pair by pair."""
    left, out = list(sections), []
    for i in range(sum(sections)):
        if order == "blocks":
            a = next(a for a, n in enumerate(left) if n)
        else:
            a = i % len(left)
            a = a if i // len(left) < sections[a] else 0
        left[a] -= 1
        out.append(a)
    assert not any(left)
    return np.array(out)


def rotate(x, pos, axis, table, layout):
    """x [T, H, D] in its own precision."""
    y, n = x.copy(), table.shape[1]
    for i in range(n):
        p, q = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = (table[pos[axis[i]], i, j].astype(x.dtype)[:, None] for j in (0, 1))
        y[:, :, p] = x[:, :, p] * c - x[:, :, q] * s
        y[:, :, q] = x[:, :, q] * c + x[:, :, p] * s
    return y


CASES = [  # T, H, D, sections, order, layout, in, out
    (1, 72, 128, (16, 24, 24), "blocks", "half", "f32", "bf16"), (5, 3, 128, (24, 20, 20), "turns", "half", "bf16", "bf16"),
    (7, 2, 64, (8, 12, 12), "blocks", "interleaved", "f16", "f32"), (9, 4, 80, (20, 20), "blocks", "half", "f16", "f16"),
    (33, 5, 128, (11, 11, 10), "turns", "interleaved", "f32", "f16"), (4, 2, 96, (6, 5, 5), "turns", "half", "f32", "f32"),
    (3, 3, 50, (2, 1), "blocks", "half", "bf16", "f32"), (6, 1, 64, (0, 32), "blocks", "half", "f32", "f32"),
    (6, 2, 64, (10, 6, 2, 6), "turns", "half", "f16", "bf16"), (2, 2, 1024, (200, 156, 156), "blocks", "interleaved", "f32", "f32"),
    (2, 2, 1024, (129, 128, 128, 127), "turns", "half", "f16", "f16"), (3, 2, 64, (32,), "blocks", "half", "f32", "f32"),
    (3, 2, 64, (32,), "turns", "half", "f32", "f32"), (2000, 72, 128, (24, 20, 20), "turns", "half", "bf16", "bf16"),
    (45000, 3, 64, (8, 8), "blocks", "half", "bf16", "f16"), (1900, 71, 128, (16, 24, 24), "blocks", "half", "f16", "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("view", ["dense", "odd"])
def test_axes(case, view):
    T, H, D, sections, order, layout, src, dst = case
    torch = torch_cuda()
    r = np.random.default_rng(T * 100 + D)
    P, half = 300, sum(sections)
    whole = torch.from_numpy(r.normal(0, 2, (T, H + 2, D + 3)).astype(np.float32)).cuda().to(ref.torch_dtype(torch, src))
    x = whole[:, :H, :D].contiguous() if view == "dense" else whole[:, 1:1 + H, 1:1 + D]
    pos = r.integers(0, P, (len(sections), T))
    tab = ref.rope_table(P, 2 * half).astype(np.float32)
    xf, axis = x.float().cpu().numpy(), axis_of(sections, order)
    say("axes", case, view)
    kw = dict(layout=layout, sections=sections, order=order)
    got = cla.rope(x, ints(pos), torch.from_numpy(tab).cuda(), out_dtype=ref.torch_dtype(torch, dst), **kw)
    want = torch.from_numpy(rotate(xf, pos, axis, tab, layout)).to(ref.torch_dtype(torch, dst))
    assert np.array_equal(bits(got), bits(want))
    if T < 100:
        exact = rotate(xf.astype(np.float64), pos, axis, tab, layout)
        err = np.abs(got.double().cpu().numpy() - exact)
        # two products and a sum in fp32 (of at most twice the largest input), then one rounding
        assert (err <= ref.U[dst] * np.abs(exact) * 1.001 + 4 * 2.0 ** -24 * 2 * np.abs(xf).max()).all()
    if src == dst:  # in place
        assert cla.rope(x, ints(pos), torch.from_numpy(tab).cuda(), out=x, **kw) is x
        assert np.array_equal(bits(x), bits(want))


def test_equal_axes_are_one():
    torch = torch_cuda()
    x = torch.randn(50, 6, 128, device="cuda")
    pos = ints(np.arange(50) * 3)
    table = cla.rope_table(200, 128, scaling="yarn", factor=4.0, trained=64)
    one = cla.rope(x, pos, table)
    for sections, order in (((16, 24, 24), "blocks"), ((24, 20, 20), "turns"), ((64,), "blocks"), ((30, 34), "blocks")):
        same = pos[None].expand(len(sections), 50).contiguous()
        assert torch.equal(cla.rope(x, same, table, sections=sections, order=order), one)
    # frequencies that start anew: each section is a rotation of its own
    sections = (12, 20)
    pos = torch.stack([pos, pos.flip(0)])
    table = torch.cat([cla.rope_table(200, 2 * n) for n in sections], 1).contiguous()
    x = x[:, :, :64].contiguous()
    got = cla.rope(x, pos, table, layout="interleaved", sections=sections)
    for at, n, p in ((0, 12, pos[0]), (24, 20, pos[1])):
        part = x[:, :, at:at + 2 * n].contiguous()
        assert torch.equal(got[:, :, at:at + 2 * n], cla.rope(part, p.contiguous(), cla.rope_table(200, 2 * n), layout="interleaved"))


def test_positions_outside_the_table():
    torch = torch_cuda()
    for D, sections in ((64, (16, 8, 8)), (24, (6, 3, 3)), (128, (16, 24, 24))):
        x = torch.ones(4, 2, D, device="cuda")
        half = sum(sections)
        table = cla.rope_table(10, 2 * half)
        pos = np.array([[0, 10, 1, 9], [0, 3, -1, 9], [0, 2, 10, 9]])
        y = cla.rope(x, ints(pos), table, sections=sections).cpu().numpy()
        axis = axis_of(sections, "blocks")
        bad = (pos < 0) | (pos >= 10)
        want = np.concatenate([bad[axis], bad[axis]]).T  # [T, D]
        assert np.array_equal(np.isnan(y), np.repeat(want[:, None], 2, 1))


APPEND = [(1, 8, 128, "int8", "f32", (16, 24, 24), "blocks", "half"), (37, 5, 128, "int4", "bf16", (24, 20, 20), "turns", "half"),
          (20, 3, 64, "int8", "f16", (8, 4, 4), "blocks", "interleaved"), (9, 2, 64, "int4", "f32", (5, 4), "turns", "half"),
          (300, 16, 128, "int8", "bf16", (0, 40, 24), "blocks", "half"), (12, 1, 64, "int8", "f32", (9, 0, 1, 1), "blocks", "interleaved")]


@pytest.mark.parametrize("case", APPEND, ids=str)
@pytest.mark.parametrize("view", ["dense", "odd"])
def test_append(case, view):
    T, H, D, kind, src, sections, order, layout = case
    torch = torch_cuda()
    r = np.random.default_rng(T + D)
    P, half, page = 90, sum(sections), 16
    whole = torch.from_numpy(r.normal(0, 2, (2, T, H + 1, D + 3)).astype(np.float32)).cuda().to(ref.torch_dtype(torch, src))
    k, v = whole[:, :, :H, :D].contiguous() if view == "dense" else whole[:, :, 1:, 2:2 + D]
    pos = r.integers(0, P, (len(sections), T))
    used = [a for a, n in enumerate(sections) if n]
    pos[[a for a, n in enumerate(sections) if not n]] = -5  # an axis without pairs: its positions mean nothing
    bad = np.zeros(T, bool)
    if T > 2:
        pos[used[-1], 1], pos[used[0], 2] = P, -1
        bad[[1, 2]] = True
    tab = ref.rope_table(P, 2 * half).astype(np.float32)
    cache = cla.KVCache(-(-T // page) + 2, page, H, D, kind)
    slots = r.permutation(cache.pages * page)[:T]
    say("append", case, view)
    cache.append(k, v, ints(slots), ints(pos), torch.from_numpy(tab).cuda(), layout=layout, sections=sections, order=order)
    got_k, got_v = cache.read(ints(slots), dtype=torch.float32)
    kf = rotate(k.float().cpu().numpy(), np.where((pos < 0) | (pos >= P), 0, pos), axis_of(sections, order), tab, layout)
    kf[bad] = 0
    for got, want in ((got_k, kf), (got_v, v.float().cpu().numpy())):
        q, s = ref.quantise(want, kind)
        assert np.array_equal(got.cpu().numpy(), ref.stored(q, s, kind).astype(np.float32))


def test_stream_and_graph():
    torch = torch_cuda()
    x = torch.randn(40, 6, 128, device="cuda").bfloat16()
    pos = ints(np.random.default_rng(1).integers(0, 100, (3, 40)))
    table = cla.rope_table(100, 128)
    graph = torch.cuda.CUDAGraph()
    cla.rope(x, pos, table, sections=(24, 20, 20), order="turns")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = cla.rope(x, pos, table, sections=(24, 20, 20), order="turns")
    for _ in range(3):
        x.copy_(torch.randn(40, 6, 128, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, cla.rope(x, pos, table, sections=(24, 20, 20), order="turns"))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        z = cla.rope(x, pos, table, sections=(24, 20, 20), order="turns")
    side.synchronize()
    assert torch.equal(y, z)


def test_refusals():
    torch = torch_cuda()
    x, table = torch.zeros(4, 2, 64, device="cuda"), cla.rope_table(10, 64)
    pos = ints(np.zeros((3, 4)))
    cache = cla.KVCache(4, 16, 2, 64, "int8")
    for kw in (dict(sections=(16, 16)), dict(sections=(16, 8, 8), order="other"), dict(sections=(16, 8.0, 8)), dict(sections=(33, 0, -1))):
        with pytest.raises(ValueError):
            cla.rope(x, pos, table, **kw)
        with pytest.raises(ValueError):
            cache.append(x, x, pos[0], pos, table, **kw)
    with pytest.raises(ValueError):
        cla.rope(x, pos[0], table, sections=(32,))
    with pytest.raises(ValueError):
        cla.rope(x, pos, table)
    with pytest.raises(ValueError):
        cache.append(x, x, pos[0], sections=(16, 8, 8))
    with pytest.raises(cla.ClError):
        cla.rope(x, pos, table, sections=(16, 8, 7))
    with pytest.raises(cla.ClError):  # 24 pairs have six turns of axis 1
        cla.rope(x, ints(np.zeros((4, 4))), cla.rope_table(10, 48), sections=(10, 8, 0, 6), order="turns")
