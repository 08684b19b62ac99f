"""Attention of drafted tokens over the quantised cache against a 64-bit reference (needs an MI355X).

Tolerances follow from the roundings (serving_ref.attention_tolerance), before any run.
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


class Problem:
    """A cache with garbage wherever no token lies, queries, masks, and the reference's answer."""

    def __init__(self, ctx, new, hq, hkv, D, page, kind, dtype, mask="tree", seed=0, sharp=1.0, spread=0.0, scale=None,
                 extra_width=0):
        torch = torch_cuda()
        r = np.random.default_rng(seed + 7 * D + page)
        self.torch, self.dtype, self.D, self.hq, self.hkv = torch, dtype, D, hq, hkv
        ctx, new = np.asarray(ctx), np.asarray(new)
        B, n = len(ctx), ctx + new
        self.ctx, self.new, self.n = ctx, new, n
        self.scale = 1.0 / np.sqrt(D) if scale is None else scale
        need = int((-(-n // page)).sum())
        pages = need + 2
        width = max(1, int((-(-n // page)).max(initial=1))) + extra_width
        self.cache = cla.KVCache(pages, page, hkv, D, kind)
        # what no token wrote: bytes of any kind, scales NaN and infinite
        kb = r.integers(0, 256, self.cache.k.shape).astype(np.uint8)
        vb = r.integers(0, 256, self.cache.v.shape).astype(np.uint8)
        junk = np.array([np.nan, np.inf, -np.inf, 60000.0], np.float16)
        ks, vs = (junk[r.integers(0, 4, self.cache.k_scale.shape)] for _ in range(2))
        self.table = r.integers(-2 ** 31, 2 ** 31, (B, width)).astype(np.int32)  # unused entries: anything
        order, at = r.permutation(pages), 0
        self.kv = []
        for b in range(B):
            m = int(-(-n[b] // page))
            mine = order[at:at + m]
            at += m
            self.table[b, :m] = mine
            k = r.normal(0, 1, (n[b], hkv, D)) * (1 + 4 * (r.random((1, hkv, D)) < 0.05))
            v = r.normal(0, 1, (n[b], hkv, D))
            if spread:  # heads and tokens of very different size
                v = v * np.exp(r.normal(0, spread, (n[b], hkv, 1)))
                k = k * np.exp(r.normal(0, min(spread, 1.0), (1, hkv, 1)))
            out = []
            for val, by, sc in ((k, kb, ks), (v, vb, vs)):
                q, s = ref.quantise(val.astype(np.float32), kind)
                where = (mine[np.arange(n[b]) // page], slice(None), np.arange(n[b]) % page)
                by[where], sc[where] = ref.codes_to_bytes(q, kind), s
                out.append(ref.stored(q, s, kind))
            self.kv.append(out)
        for t, a in ((self.cache.k, kb), (self.cache.v, vb), (self.cache.k_scale, ks), (self.cache.v_scale, vs)):
            t.copy_(torch.from_numpy(a))
        T = int(new.sum())
        self.q = torch.from_numpy((r.normal(0, 1, (T, hq, D)) * sharp).astype(np.float32)).cuda().to(
            ref.torch_dtype(torch, dtype))
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.max_q = int(new.max(initial=0))
        words = -(-max(self.max_q, 1) // 64)
        self.see, rows = [], []
        for b in range(B):
            t = int(new[b])
            if mask == "tree":
                m = np.zeros((t, t), bool)
                for i in range(t):
                    up = int(r.integers(-1, i)) if i else -1
                    if up >= 0:
                        m[i] = m[up]
                    m[i, i] = True
            elif mask == "none":  # sees no new token
                m = np.zeros((t, t), bool)
            elif mask == "random":
                m = r.random((t, t)) < 0.4
            else:  # chain
                m = np.tril(np.ones((t, t), bool))
            self.see.append(np.concatenate([np.ones((t, ctx[b]), bool), m], 1))
            full = np.zeros((t, 64 * words), bool)
            full[:, :t] = m
            full[:, t:] = r.random((t, 64 * words - t)) < 0.5  # bits past the new tokens mean nothing
            rows.append(np.packbits(full, axis=1, bitorder="little").reshape(t, 8 * words))
        bits = np.concatenate(rows) if rows else np.zeros((0, 8 * words), np.uint8)
        self.mask = None if mask == "chain" else torch.from_numpy(np.ascontiguousarray(bits).view(np.int64)).cuda()

    def dev(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()

    def call(self, **kw):
        args = dict(max_q=self.max_q, max_ctx=int(self.ctx.max(initial=0)), tree_mask=self.mask)
        if abs(self.scale * np.sqrt(self.D) - 1) > 1e-12:
            args["scale"] = self.scale
        args.update(kw)
        q = args.pop("q", self.q)
        return cla.tree_attention(q, self.cache, self.dev(self.table), self.dev(self.ctx), self.dev(self.cu), **args)

    def check(self, got, rows=None):
        o = got.double().cpu().numpy()
        worst = 0.0
        g = self.hq // self.hkv
        for b in range(len(self.ctx)):
            k, v = self.kv[b]
            for h in range(self.hq):
                q = self.q[self.cu[b]:self.cu[b + 1], h].double().cpu().numpy()
                want, absv, mag = ref.attention(q, k[:, h // g], v[:, h // g], self.see[b], self.scale)
                tol = ref.attention_tolerance(want, absv, mag, self.n[b], self.D, self.dtype)
                mine = o[self.cu[b]:self.cu[b + 1], h]
                err = np.abs(mine - want)
                assert (err <= tol).all(), (b, h, float((err / tol).max()), np.argwhere(~(err <= tol))[:3])
                dark = ~self.see[b].any(-1)
                assert (mine[dark] == 0).all()
                worst = max(worst, float((err / tol).max(initial=0.0)))
        return worst


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257, 511, 640]


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1), (6, 2)])
def test_single_tokens_of_every_length(kind, D, dtype, hq, hkv):
    say("lengths", kind, D, dtype, hq, hkv)
    p = Problem(LENGTHS, [1] * len(LENGTHS), hq, hkv, D, 16, kind, dtype, mask="chain", seed=hq)
    say("worst", p.check(p.call()))


TREES = [  # ctx, new, hq, hkv, D, page, kind, dtype, mask
    ([0], [1], 1, 1, 64, 16, "int8", "f16", "none"),              # nothing to see at all
    ([0, 5, 0], [3, 0, 7], 2, 1, 128, 16, "int4", "bf16", "random"),  # rows that may see nothing, a sequence without any
    ([100, 0, 33], [16, 16, 5], 8, 1, 128, 16, "int8", "bf16", "tree"),
    ([700, 1], [64, 64], 8, 1, 128, 64, "int8", "f16", "tree"),
    ([63, 200], [65, 130], 4, 2, 64, 128, "int4", "f16", "tree"),
    ([17], [256], 3, 1, 128, 32, "int8", "bf16", "random"),
    ([1000, 31], [2, 9], 52, 52, 128, 32, "int8", "f16", "tree"),
    ([300], [33], 16, 2, 64, 1024, "int4", "bf16", "chain"),
    ([2049, 5, 900], [8, 1, 3], 32, 4, 128, 256, "int4", "f16", "none"),
    ([12], [100], 1, 1, 64, 16, "int8", "bf16", "chain"),
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}over{c[3]}-{c[4]}-{c[6]}-{c[7]}-{c[8]}")
def test_trees(case):
    say("trees", case)
    p = Problem(*case[:8], mask=case[8], seed=3)
    say("worst", p.check(p.call()))
    again = p.call()
    assert p.torch.equal(p.call(), again)  # bitwise the same
    # the hint for the longest context only sizes the launch
    for hint in (0, 1, 100000, None):
        p.check(p.call(max_ctx=hint))


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask,dtype,spread", [("tree", "f16", 0.0), ("random", "bf16", 2.0), ("chain", "f16", 2.0),
                                               ("none", "bf16", 0.0)])
def test_many_rows_of_a_kv_head(kind, D, mask, dtype, spread):
    # up to 520 rows that read the same keys, sequences with fewer rows and keys than the launch was sized for
    p = Problem([5000, 0, 77, 31, 700], [65, 17, 33, 1, 16], 16, 2, D, 32, kind, dtype, mask=mask, seed=31, spread=spread)
    say("many rows", kind, D, mask, p.check(p.call()))
    assert p.torch.equal(p.call(), p.call())
    clean = p.call()
    q = p.q.clone()
    q[2, 1] = float("nan")
    got = p.call(q=q)
    assert got[2, 1].isnan().all()
    got[2, 1] = clean[2, 1]
    assert p.torch.equal(got, clean)
    keep = p.table.copy()
    p.table[0, 3] = p.cache.pages  # in the old tokens of the first sequence: every row sees it
    got = p.call()
    p.table = keep
    assert got[:65].isnan().all() and p.torch.equal(got[65:], clean[65:])


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,hint,mask,dtype,spread", [
    (29000, 64, 29000, "tree", "bf16", 0.0), (5000, 65, 120000, "random", "f16", 2.0), (0, 200, 100000, "random", "bf16", 0.0),
    (77, 16, 250000, "chain", "f16", 2.0), (700, 33, 100000, "none", "bf16", 2.0)])
def test_many_rows_of_one_sequence(kind, D, ctx, new, hint, mask, dtype, spread):
    # 128 rows to a workgroup; a hint that is too long sizes the launch as if the sequence were
    p = Problem([ctx], [new], 16, 2, D, 32, kind, dtype, mask=mask, seed=37, spread=spread)
    clean = p.call(max_ctx=hint)
    say("many rows of one", kind, D, ctx, new, p.check(clean))
    assert p.torch.equal(p.call(max_ctx=hint), clean)
    q = p.q.clone()
    q[2, 1] = float("nan")
    got = p.call(q=q, max_ctx=hint)
    assert got[2, 1].isnan().all()
    got[2, 1] = clean[2, 1]
    assert p.torch.equal(got, clean)
    if ctx >= 77:
        p.table[0, 1] = p.cache.pages  # in the old tokens: every row sees it
        assert p.call(max_ctx=hint).isnan().all()


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,hq,hkv", [
    ([4700] + [37 * i % 700 for i in range(23)], [5, 4, 0, 1] * 6, 16, 2),  # up to 40 rows, in groups of 32
    ([4700] + [0] * 23, [5] + [1] * 23, 16, 2),
    ([600, 90, 2000], [7, 16, 3], 32, 4),                                   # up to 128, in groups of 16
    ([3700, 100], [13, 16], 64, 8),                                         # fewer than 128
    ([29000], [16], 8, 1),                                                  # 128, in groups of 32 or at once
    ([20, 31, 0, 5, 17], [1, 1, 2, 3, 1], 8, 4),                            # a wavefront each: one block of keys
    ([200 - 5 * i for i in range(40)], [1 + i % 5 for i in range(40)], 64, 32),  # the same: many cells of few keys
    ([60] * 18, [17, 9, 30] * 6, 64, 8),
], ids=["groups32", "groups32-short", "groups16", "many-cells", "long", "one-block", "few-keys", "few-keys-rows"])
def test_row_groups(kind, D, ctx, new, hq, hkv):
    p = Problem(ctx, new, hq, hkv, D, 64, kind, "bf16", mask="tree", seed=41, spread=1.0)
    say("row groups", kind, D, hq, hkv, p.check(p.call()))
    assert p.torch.equal(p.call(), p.call())
    p.check(p.call(max_ctx=0))         # few, long chunks
    p.check(p.call(max_ctx=10 * max(ctx)))  # more rows to a workgroup than these lengths would get


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_contexts(kind, dtype):
    p = Problem([9001, 40, 20003], [1, 3, 5], 8, 2, 128, 64, kind, dtype, seed=11)
    say("long", kind, dtype, p.check(p.call()))


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("dtype,sharp,spread", [("f16", 12.0, 0.0), ("bf16", 3e4, 0.0), ("f16", 1e-4, 3.0), ("bf16", 1.0, 3.0),
                                                ("f16", 3.0, 2.0), ("bf16", 1e-20, 0.0), ("f16", 0.0, 0.0)])
def test_scores_and_values_of_very_different_size(kind, dtype, sharp, spread):
    # one key takes everything; nearly uniform weights; scales of V that span orders of magnitude
    p = Problem([1500, 77], [4, 9], 8, 2, 128, 32, kind, dtype, seed=21, sharp=sharp, spread=spread)
    say("sizes", kind, dtype, sharp, spread, p.check(p.call()))


@pytest.mark.parametrize("new", [1, 40])
def test_pages_past_4_gib(new):
    torch = torch_cuda()
    r = np.random.default_rng(23)
    pages, page, H, D, n = 4300, 1024, 8, 128, 1500  # 4.5 GB of keys
    cache = cla.KVCache(pages, page, H, D, "int8")
    table = np.array([[pages - 1, pages - 30]], np.int32)
    slots = table[0][np.arange(n) // page] * page + np.arange(n) % page
    k, v = (torch.from_numpy(r.normal(0, 1, (n, H, D)).astype(np.float32)).cuda() for _ in range(2))
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    cache.append(k, v, dev(slots))
    ks, vs = (x.double().cpu().numpy() for x in cache.read(dev(slots), dtype=torch.float32))
    q = torch.from_numpy(r.normal(0, 1, (new, 2 * H, D)).astype(np.float32)).cuda().half()
    say("past 4 GiB", new)
    got = cla.tree_attention(q, cache, dev(table), dev([n - new]), dev([0, new]), max_q=new).double().cpu().numpy()
    see = np.concatenate([np.ones((new, n - new), bool), np.tril(np.ones((new, new), bool))], 1)
    for h in range(2 * H):
        want, absv, mag = ref.attention(q[:, h].double().cpu().numpy(), ks[:, h // 2], vs[:, h // 2], see, 1 / np.sqrt(D))
        assert (np.abs(got[:, h] - want) <= ref.attention_tolerance(want, absv, mag, n, D, "f16")).all(), h


def test_scale_argument_and_strided_queries():
    for scale in (0.0, -0.05, 1.0):
        p = Problem([130], [6], 4, 2, 64, 16, "int8", "f16", seed=2, scale=scale)
        p.check(p.call())
    p = Problem([130, 9], [6, 2], 6, 2, 128, 16, "int8", "bf16", seed=2)
    wide = p.torch.zeros(p.q.shape[0], 10, 128, dtype=p.q.dtype, device="cuda")
    wide[:, 3:9] = p.q
    assert p.torch.equal(p.call(q=wide[:, 3:9]), p.call())
    odd = p.torch.zeros(p.q.shape[0], 6, 131, dtype=p.q.dtype, device="cuda")
    odd[..., 1:129] = p.q
    assert p.torch.equal(p.call(q=odd[..., 1:129]), p.call())
    out = p.torch.empty_like(p.q)
    assert p.call(out=out) is out and p.torch.equal(out, p.call())


def test_bad_rows_stay_alone():
    # a query of NaN, one of infinities, and a page outside the cache touch their own rows only
    p = Problem([100, 100], [5, 5], 4, 2, 128, 16, "int8", "f16", seed=4)
    clean = p.call()
    q = p.q.clone()
    q[2, 1] = float("nan")
    q[3, 0, 5] = float("inf")
    got = p.call(q=q)
    assert got[2, 1].isnan().all() and got[3, 0].isnan().all()
    touched = p.torch.zeros(10, 4, dtype=p.torch.bool, device="cuda")
    touched[2, 1] = touched[3, 0] = True
    assert p.torch.equal(got[~touched], clean[~touched])
    for page in (-1, p.cache.pages, 2 ** 31 - 1):
        keep = p.table.copy()
        p.table[1, 2] = page
        got = p.call()
        p.table = keep
        assert p.torch.equal(got[:5], clean[:5]) and got[5:].isnan().all()
    # a sequence longer than its row of the block table
    ctx = p.ctx.copy()
    p.ctx = np.array([100, 5000])
    got = p.call(max_ctx=5000)
    p.ctx = ctx
    assert p.torch.equal(got[:5], clean[:5]) and got[5:].isnan().all()


def test_sequences_that_do_not_fit_are_left_out():
    p = Problem([50, 60, 70], [2, 3, 4], 2, 1, 64, 16, "int8", "f16", seed=6, mask="chain")
    clean = p.call()
    out = p.torch.full_like(clean, 9.0)
    p.call(out=out, max_q=3)  # the last sequence has 4 new tokens
    assert p.torch.equal(out[:5], clean[:5]) and (out[5:] == 9.0).all()


def test_other_stream_and_graph():
    p = Problem([400, 33, 1200], [4, 1, 7], 8, 2, 128, 32, "int8", "bf16", seed=8)
    torch = p.torch
    want = p.call()
    tab, ctx, cu = p.dev(p.table), p.dev(p.ctx), p.dev(p.cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=p.max_q, max_ctx=1200, tree_mask=p.mask)
    s.synchronize()
    assert torch.equal(got, want)
    q = p.q.clone()
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cla.tree_attention(q, p.cache, tab, ctx, cu, max_q=p.max_q, max_ctx=1200, tree_mask=p.mask, out=out)
    for i in range(4):
        q.copy_(p.q * (1.0 + i))
        eager = cla.tree_attention(q, p.cache, tab, ctx, cu, max_q=p.max_q, max_ctx=1200, tree_mask=p.mask)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_first_call_recorded():
    # a cache whose first calls are recorded: their workspaces are cleared by the replays, so nobody else may have them
    p = Problem([400, 33], [4, 1], 8, 2, 128, 32, "int8", "bf16", seed=18)
    torch = p.torch
    want = p.call()
    tab, ctx, cu = p.dev(p.table), p.dev(p.ctx), p.dev(p.cu)
    fresh = cla.KVCache(kind="int8", k=p.cache.k, v=p.cache.v, k_scale=p.cache.k_scale, v_scale=p.cache.v_scale)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(2):
                cla.tree_attention(p.q, fresh, tab, ctx, cu, max_q=p.max_q, max_ctx=400, tree_mask=p.mask, out=out)
        graphs.append((g, out))
    assert len(fresh._work) == 2
    with torch.cuda.stream(s):
        eager = cla.tree_attention(p.q, fresh, tab, ctx, cu, max_q=p.max_q, max_ctx=400, tree_mask=p.mask)
    s.synchronize()
    assert torch.equal(eager, want)
    for _ in range(3):
        for g, out in reversed(graphs):
            out.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    for x in (p.cache, fresh):  # a workspace to a stream
        with torch.cuda.stream(s):
            got = cla.tree_attention(p.q, x, tab, ctx, cu, max_q=p.max_q, max_ctx=400, tree_mask=p.mask)
        s.synchronize()
        assert torch.equal(got, want)
    assert len({a for a, _ in p.cache._work.values()}) == len(p.cache._work) == 2


def test_refusals():
    p = Problem([40], [3], 4, 2, 64, 16, "int8", "f16", seed=9)
    torch = p.torch
    tab, ctx, cu = p.dev(p.table), p.dev(p.ctx), p.dev(p.cu)
    ok = dict(max_q=3, max_ctx=40, tree_mask=p.mask)
    for bad in (lambda: cla.tree_attention(p.q.float(), p.cache, tab, ctx, cu, **ok),
                lambda: cla.tree_attention(p.q[..., :32], p.cache, tab, ctx, cu, **ok),
                lambda: cla.tree_attention(p.q, p.cache, tab.long(), ctx, cu, **ok),
                lambda: cla.tree_attention(p.q, p.cache, tab[:0], ctx, cu, **ok),
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu[:1], **ok),
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=3, tree_mask=p.mask[:2]),
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=3, tree_mask=p.mask.int()),
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=3, out=p.q[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cla.tree_attention(p.q[:, :3].contiguous(), p.cache, tab, ctx, cu, **ok),  # 3 heads over 2
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=257),
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=65, tree_mask=p.mask),  # one word
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=3, max_ctx=-1),
                lambda: cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=3, scale=float("nan"))):
        with pytest.raises(cla.ClError):
            bad()
    assert cla.tree_attention(p.q[:0], p.cache, tab, ctx, torch.zeros_like(cu), max_q=3).shape == (0, 4, 64)
