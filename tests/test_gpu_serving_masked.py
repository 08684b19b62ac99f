"""Attention with memory behind the mask that no token was ever written to (needs an MI355X).

A new token that no row sees (padding of a tree, stored with slot -1) and a tile without a page leave whatever is in
memory as a key's codes and scales; rows that do not see it must come out as if it were not there.  Tolerances are
serving_ref.attention_tolerance's, which counts only tokens that a row sees.
"""
import sys

import pytest

from test_gpu_serving_attention import Problem

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def hide(p, b, tokens):
    """No row of sequence b sees its new tokens `tokens` any more."""
    for t in tokens:
        p.see[b][:, p.ctx[b] + t] = False
        bit = (1 << t % 64) - (1 << 64 if t % 64 == 63 else 0)
        p.mask[p.cu[b]:p.cu[b + 1], t // 64] &= ~bit


def place(p, b, j):
    """Page and place of cached token j of sequence b."""
    return int(p.table[b, j // p.cache.page_size]), j % p.cache.page_size


def junk(p, b, tokens, scale, code):
    for t in tokens:
        page, o = place(p, b, int(p.ctx[b]) + t)
        p.cache.k[page, :, o] = code
        p.cache.v[page, :, o] = code
        p.cache.k_scale[page, :, o] = scale
        p.cache.v_scale[page, :, o] = scale


# ctx, new, q heads, kv heads: one wavefront, four with 16 rows, with 32, and 128 rows to a workgroup
SHAPES = [([20, 0, 5], [9, 12, 3], 4, 4), ([300, 70], [7, 5], 6, 2), ([5000, 0, 77, 700], [65, 17, 33, 16], 16, 2),
          ([29000], [64], 16, 2)]


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=["wave", "rows16", "rows32", "rows128"])
@pytest.mark.parametrize("scale,code", [(float("nan"), 0), (float("inf"), 255), (float("-inf"), 7), (60000.0, 0), (8192.0, 0)])
def test_new_tokens_that_no_row_sees(kind, D, shape, scale, code):
    ctx, new, hq, hkv = shape
    p = Problem(ctx, new, hq, hkv, D, 32, kind, "f16", mask="tree", seed=51)
    say("hidden", kind, D, shape, scale, code)
    for b, t in enumerate(new):
        gone = list(range(1, t, 3))
        hide(p, b, gone)
        junk(p, b, gone, scale, code)
    got = p.call()
    say("worst", p.check(got))
    # and bit for bit what there is without them
    for b, t in enumerate(new):
        junk(p, b, range(1, t, 3), 0.0, 0x88)
    assert p.torch.equal(p.call(), got)


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,hq,hkv", [([32], [40], 4, 4), ([320, 17], [40, 3], 16, 2), ([28992], [64], 16, 2)])
def test_page_that_only_later_tokens_see(kind, D, ctx, new, hq, hkv):
    # a chain: tokens before the page's first do not see it, the others are NaN
    p = Problem(ctx, new, hq, hkv, D, 16, kind, "bf16", mask="chain", seed=53)
    # page 0, which is read in place of a bad one, holds nothing
    used = {int(x) for b in range(len(ctx)) for x in p.table[b, :-(-int(p.n[b]) // 16)]}
    free = next(i for i in range(p.cache.pages) if i not in used)
    if 0 in used:
        for t in (p.cache.k, p.cache.v, p.cache.k_scale, p.cache.v_scale):
            t[free] = t[0]
        p.table[p.table == 0] = free
    p.cache.k_scale[0], p.cache.v_scale[0] = float("nan"), float("inf")
    clean = p.call()
    say("page", kind, D, ctx, p.check(clean))
    at = ctx[0] // 16 + 1  # its tokens are new tokens 16 .. 31 of the first sequence
    for page in (-1, p.cache.pages):
        p.table[0, at] = page
        got = p.call()
        assert p.torch.equal(got[:16], clean[:16]) and got[16:new[0]].isnan().all()
        assert p.torch.equal(got[new[0]:], clean[new[0]:])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,hq,hkv", [([50], [12], 4, 4), ([300, 70], [30, 5], 16, 2), ([29000], [64], 16, 2)])
def test_large_values_that_other_rows_see(D, ctx, new, hq, hkv):
    # a row keeps its bits whatever the values of tokens that only other rows see (int8: their scales)
    p = Problem(ctx, new, hq, hkv, D, 32, "int8", "f16", mask="tree", seed=57)
    last = new[0] - 1
    p.see[0][:, ctx[0] + 3] = False
    p.mask[:new[0], 0] &= ~(1 << 3)
    p.see[0][last, ctx[0] + 3] = True
    p.mask[last, last // 64] |= 1 << 3
    page, o = place(p, 0, ctx[0] + 3)
    keep = p.cache.v_scale[page, :, o].clone()
    clean = p.call()
    say("large", D, ctx, p.check(clean))
    p.cache.v_scale[page, :, o] = 30000.0
    got = p.call()
    assert p.torch.equal(got[:last], clean[:last]) and p.torch.equal(got[new[0]:], clean[new[0]:])
    p.cache.v_scale[page, :, o] = keep
    assert p.torch.equal(p.call(), clean)
