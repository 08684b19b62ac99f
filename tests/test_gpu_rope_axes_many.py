"""Rotary positions with several axes for many tokens, whose cosines and sines are gathered once for a token's heads (needs an MI355X).

That is from 2^14 heads of tokens on at aligned heads, but for fp32 inputs of 2^17 and more.  Bit by bit in fp32.
"""
import sys

import numpy as np
import pytest

import compressed_linear_amd as cla
import serving_ref as ref
from gpu_util import torch_cuda
from test_gpu_rope_axes import axis_of, bits, ints

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def rotated(x, pos, axis, table, layout):
    """x [T, H, D] float32 with the table's row of each pair's axis; NaN where that position is outside."""
    half = table.shape[1]
    p = pos[axis].T  # [T, half]
    out = (p < 0) | (p >= len(table))
    cs = table[np.where(out, 0, p), np.arange(half)]  # [T, half, 2]
    cs[out] = np.nan
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


CASES = [  # T, H, D, sections, order, layout, in, out
    (1901, 9, 128, (24, 20, 20), "turns", "interleaved", "bf16", "bf16"),
    (2051, 8, 128, (16, 24, 24), "blocks", "interleaved", "f32", "f32"),       # 2^14 to 2^17 in fp32
    (2051, 8, 128, (24, 20, 20), "turns", "half", "f32", "bf16"),
    (701, 72, 128, (16, 8, 8), "blocks", "interleaved", "f16", "f32"),         # half of a head is rotated
    (6007, 3, 64, (9, 7), "turns", "half", "f32", "f16"),
    (701, 72, 80, (11, 10, 3), "blocks", "half", "bf16", "f32"),
    (8193, 16, 64, (12, 10, 10), "turns", "interleaved", "f32", "f32"),        # past 2^17 in fp32: the kernel of few tokens
    (8193, 16, 64, (12, 10, 10), "blocks", "half", "f32", "bf16"),
    (8191, 16, 64, (12, 10, 10), "blocks", "half", "f32", "f32"),              # and just below
    (8193, 16, 64, (12, 10, 10), "turns", "interleaved", "f16", "f16"),
    (301, 56, 1024, (129, 128, 128, 127), "turns", "half", "f16", "f16"),      # two tokens' cosines and sines fill LDS
    (301, 56, 1024, (200, 156, 0, 156), "blocks", "interleaved", "bf16", "f32"),
    (20001, 1, 16, (8, 0), "blocks", "interleaved", "bf16", "bf16"),
    (40, 500, 64, (0, 16), "blocks", "half", "f16", "f16"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("outside", [False, True], ids=["inside", "outside"])
def test_many_tokens(case, outside):
    T, H, D, sections, order, layout, src, dst = case
    torch = torch_cuda()
    r = np.random.default_rng(T + D)
    P, half = 300, sum(sections)
    whole = torch.from_numpy(r.normal(0, 2, (T, H + 2, D)).astype(np.float32)).cuda().to(ref.torch_dtype(torch, src))
    pos = r.integers(0, P, (len(sections), T))
    if outside:
        at = r.random(pos.shape) < 0.1
        pos[at] = r.choice([-1, P, -2 ** 31, 2 ** 31 - 1, P + 7], int(at.sum()))
    tab = ref.rope_table(P, 2 * half).astype(np.float32)
    table, axis = torch.from_numpy(tab).cuda(), axis_of(sections, order)
    kw = dict(layout=layout, sections=sections, order=order)
    for x in (whole[:, :H].contiguous(), whole[:, 1:1 + H]):  # dense, and heads of wider tokens
        want = torch.from_numpy(rotated(x.float().cpu().numpy(), pos, axis, tab, layout)).to(ref.torch_dtype(torch, dst))
        nan = torch.isnan(want).numpy()
        assert nan.any() == (outside and any(sections))
        say("many", case, outside, x.stride())
        got = cla.rope(x, ints(pos), table, out_dtype=want.dtype, **kw)
        assert np.array_equal(torch.isnan(got).cpu().numpy(), nan)
        assert np.array_equal(np.where(nan, 0, bits(got)), np.where(nan, 0, bits(want)))
        if src == dst:  # in place
            assert cla.rope(x, ints(pos), table, out=x, **kw) is x
            assert np.array_equal(bits(x), bits(got))


def test_many_tokens_in_a_graph():
    torch = torch_cuda()
    x = torch.randn(2048, 9, 128, device="cuda").bfloat16()
    pos = ints(np.random.default_rng(1).integers(0, 100, (3, 2048)))
    table = cla.rope_table(100, 128)
    kw = dict(sections=(24, 20, 20), order="turns", layout="interleaved")
    cla.rope(x, pos, table, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cla.rope(x, pos, table, **kw)
    for _ in range(3):
        x.copy_(torch.randn(2048, 9, 128, device="cuda").bfloat16())
        y.zero_()
        graph.replay()
        eager = cla.rope(x, pos, table, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
