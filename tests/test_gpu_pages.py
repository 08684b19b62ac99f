"""The pages of a cache against a plain model, and the moves inside a cache that follow (needs an MI355X).

Everything here is whole numbers and copied bytes: results are equal or wrong.
"""
import sys

import numpy as np
import pytest

import compressed_linear_amd as cla
import pages_ref as ref
import serving_ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def ints(a):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def same(pool, model):
    assert np.array_equal(pool.lens.cpu().numpy(), model.lens)
    assert np.array_equal(pool.block_table.cpu().numpy(), model.table)
    assert np.array_equal(pool.refs.cpu().numpy(), model.refs)


def both(pool, model, name, *args):
    """One operation on both; their answers are equal, and so are the pools."""
    got = getattr(pool, name)(*(ints(a) if isinstance(a, (list, np.ndarray)) else a for a in args))
    want = getattr(model, name)(*args)
    if want is not None:
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy(), w), name
    if name == "extend":
        assert int(pool.left_out) == model.left_out
    same(pool, model)
    return got


def cu_of(counts):
    return np.concatenate([[0], np.cumsum(counts)])


POOLS = [  # pages, page size, sequences, width
    (1, 16, 1, 1), (7, 16, 3, 4), (100, 16, 5, 30), (50, 64, 9, 7), (333, 32, 40, 12), (3000, 16, 64, 70), (20000, 16, 130, 200),
    (40000, 16, 1500, 33), (9001, 32, 4096, 9), (17000, 128, 3, 6000),
]


@pytest.mark.parametrize("pages,page,B,width", POOLS)
def test_random_programs(pages, page, B, width):
    r = np.random.default_rng(pages + B)
    pool, model = cla.PagePool(pages, page, B, width), ref.Pool(pages, page, B, width)
    same(pool, model)
    for step in range(14 if B < 1000 else 7):
        what = ["extend", "extend", "fork", "truncate", "compact"][r.integers(5)] if step else "extend"
        if step == 0:
            counts = r.integers(0, max(2, int(1.2 * min(width, pages / B) * page)), B)
        else:
            counts = r.integers(0, [2, 5, 40, 3 * page][r.integers(4)], B) * (r.random(B) < 0.8)
        say(what, step, pages, page, B, width, int(counts.sum()))
        if what == "extend":
            cu = cu_of(counts)
            both(pool, model, what, cu, int(cu[-1]) + int(r.integers(0, 3)))
        elif what == "fork":
            parents = np.arange(B)
            some = r.random(B) < 0.5
            parents[some] = r.integers(-1, B, int(some.sum()))
            both(pool, model, what, parents)
        elif what == "truncate":
            both(pool, model, what, np.where(r.random(B) < 0.4, r.integers(-1, np.maximum(model.lens, 1) + 3), -1))
        else:
            both(pool, model, what, int(r.integers(0, [3, pages + 5][r.integers(2)])))


def test_last_page_of_several():
    # 5 tokens in 16: sequences 0 to 3 share the page; of those that are extended all copy it unless nobody else is left
    for extended in ([1, 1, 1, 1], [0, 1, 0, 1], [1, 0, 0, 0], [0, 0, 0, 2]):
        pool, model = cla.PagePool(20, 16, 6, 4), ref.Pool(20, 16, 6, 4)
        both(pool, model, "extend", cu_of([5, 0, 0, 0, 0, 0]), 5)
        both(pool, model, "fork", [0, 0, 0, 0, -1, -1])
        counts = extended + [3, 0]
        _, src, _ = both(pool, model, "extend", cu_of(counts), sum(counts))
        assert (src.cpu().numpy() >= 0).sum() == (3 if sum(extended) == 4 else sum(v > 0 for v in extended))
    # a page that is shared and full is not copied; cut into, it is
    pool, model = cla.PagePool(20, 16, 2, 4), ref.Pool(20, 16, 2, 4)
    both(pool, model, "extend", cu_of([32, 0]), 32)
    both(pool, model, "fork", [0, 0])
    _, src, _ = both(pool, model, "extend", cu_of([1, 1]), 2)
    assert (src == -1).all()
    both(pool, model, "truncate", [20, 32])
    _, src, _ = both(pool, model, "extend", cu_of([1, 0]), 1)
    assert src.tolist() == [1, -1]


def test_too_few_pages():
    # the first that does not fit is left out, and whoever comes after; what was there stays
    for pages in range(1, 12):
        pool, model = cla.PagePool(pages, 16, 5, 4), ref.Pool(pages, 16, 5, 4)
        both(pool, model, "extend", cu_of([20, 10, 0, 40, 1]), 71)
        both(pool, model, "fork", [0, 1, 0, 1, 4])
        both(pool, model, "extend", cu_of([1, 7, 14, 30, 16]), 68)
        both(pool, model, "extend", cu_of([0, 1, 0, 0, 0]), 1)
    # a table too narrow; positions that do not fit
    pool, model = cla.PagePool(30, 16, 3, 2), ref.Pool(30, 16, 3, 2)
    both(pool, model, "extend", cu_of([33, 32, 1]), 66)
    both(pool, model, "extend", [0, 2, 1, 9], 4)
    both(pool, model, "extend", [0, -3, 1, 2], 4)
    assert model.left_out == 2
    both(pool, model, "extend", [0, 0, 0, 0], 0)


def test_many_tokens():
    # more than the pages' own workgroup writes slots of
    pool, model = cla.PagePool(5000, 16, 7, 1400), ref.Pool(5000, 16, 7, 1400)
    both(pool, model, "extend", cu_of([20000, 0, 3, 9000, 1, 22399, 5000]), 56403 + 5)
    both(pool, model, "fork", [0, 0, 0, 3, 4, 5, 6])
    both(pool, model, "extend", cu_of([2300, 2500, 100, 50000, 20, 1, 3000]), 57921)  # the fourth is too long
    both(pool, model, "extend", [0, 5000, 4000, 4100, 4200, 4300, 70000, 70000], 60000)


def test_refs_at_odd_addresses_and_held_pages():
    torch = torch_cuda()
    room = torch.zeros(1001, dtype=torch.int32, device="cuda")
    pool = cla.PagePool(page_size=32, block_table=torch.full((4, 9), -1, dtype=torch.int32, device="cuda"),
                        lens=torch.zeros(4, dtype=torch.int32, device="cuda"), refs=room[1:])
    model = ref.Pool(1000, 32, 4, 9)
    pool.refs[0] += 1  # a page that the program holds itself
    model.refs[0] += 1
    both(pool, model, "extend", cu_of([100, 3, 64, 250]), 417)
    both(pool, model, "truncate", [0, -1, 10, 40])
    both(pool, model, "compact", 1000)
    assert model.refs[0] == 1 and room[0] == 0
    # taken over by another pool object
    again = cla.PagePool(page_size=32, block_table=pool.block_table, lens=pool.lens, refs=pool.refs)
    both(again, model, "extend", cu_of([1, 1, 1, 1]), 4)
    same(pool, model)


def test_a_million_pages():
    pages = 1 << 20
    pool, model = cla.PagePool(pages, 16, 3, 300000), ref.Pool(pages, 16, 3, 300000)
    say("a million pages")
    cu = cu_of([4000000, 4700000, 3])
    pool.extend(ints(cu), int(cu[-1]))
    assert int(pool.left_out) == 0
    pool.truncate(ints([16 * 200000, -1, 0]))
    model.table[0, :200000] = np.arange(200000)
    model.table[1, :293750] = np.arange(250000, 543750)
    model.lens[:] = [3200000, 4700000, 0]
    model.refs[:200000] = model.refs[250000:543750] = 1
    same(pool, model)
    src, dst = pool.compact(60000)
    want = np.arange(543749, 543749 - 50000, -1)
    assert np.array_equal(src[:50000].cpu().numpy(), want) and np.array_equal(dst[:50000].cpu().numpy(), np.arange(200000, 250000))
    assert (src[50000:] == -1).all() and (dst[50000:] == -1).all()
    to = np.arange(pages)
    to[want] = np.arange(200000, 250000)
    model.table = np.where(model.table >= 0, to[model.table], -1)
    model.refs[:] = 0
    model.refs[:493750] = 1
    same(pool, model)


# ------------------------------------------------------------------ the cache
def cache_of(pages, page, heads, dim, kind, seed=0):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = cla.KVCache(pages, page, heads, dim, kind)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (c.k_scale, c.v_scale):  # any bits
        t.view(torch.int16).copy_(torch.randint(-32768, 32767, t.shape, generator=g, device="cuda").short())
    return c


def parts(c):
    torch = torch_cuda()
    return [t.view(torch.int16 if t.element_size() == 2 else torch.uint8) for t in (c.k, c.v, c.k_scale, c.v_scale)]


CACHES = [(30, 16, 1, 64, "int4"), (30, 16, 3, 128, "int8"), (40, 64, 8, 128, "int8"), (25, 128, 5, 64, "int8"), (20, 1024, 2, 128, "int4"),
          (12, 32, 52, 128, "int4")]


@pytest.mark.parametrize("shape", CACHES, ids=str)
def test_copy_pages(shape):
    torch = torch_cuda()
    c = cache_of(*shape)
    n = shape[0]
    before = [t.clone() for t in parts(c)]
    src, dst = [1, -1, 3, n - 1, 5, 6, n, 8, -7], [n - 2, 4, 2, 0, -1, n, 9, 8, 10]
    say("copy", shape)
    c.copy_pages(ints(src), ints(dst))
    for t, old in zip(parts(c), before):
        for s, d in ((1, n - 2), (3, 2), (n - 1, 0)):
            old[d] = old[s]
        assert torch.equal(t, old)
    c.copy_pages(ints([]), ints([]))


def test_copy_more_pages_than_a_launch_has_rows():
    torch = torch_cuda()
    c = cache_of(6, 16, 1, 64, "int4")
    before = [t.clone() for t in parts(c)]
    src = torch.full((70000,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    src[3], dst[3], src[69999], dst[69999] = 2, 5, 1, 0
    c.copy_pages(src, dst)
    for t, old in zip(parts(c), before):
        old[5], old[0] = old[2], old[1]
        assert torch.equal(t, old)


@pytest.mark.parametrize("shape", CACHES, ids=str)
@pytest.mark.parametrize("most", [1, 5, 64, 256])
def test_keep(shape, most):
    torch = torch_cuda()
    pages, page, heads, dim, kind = shape
    r = np.random.default_rng(most + pages)
    B, width = 4, 5
    table = r.permutation(pages)[:B * width].reshape(B, width) if pages >= B * width else \
        np.concatenate([r.permutation(pages), np.full(B * width - pages, -1)]).reshape(B, width)
    ctx = r.integers(0, max(1, width * page - most - 2), B)
    ctx[1] = width * page - 3  # drafts past the table's end
    table[2, 3] = pages + 4    # a page that is none
    kept = r.integers(-1, most + 3, (B, most))  # any order, twice the same, past the drafts
    kept[3] = np.where(r.random(most) < 0.5, -1, kept[3])
    c = cache_of(*shape, seed=most)
    before = [t.clone() for t in parts(c)]
    say("keep", shape, most)
    c.keep(ints(table), ints(ctx), ints(kept))
    for t, old in zip(parts(c), before):
        new = old.clone()
        for b in range(B):
            for j in range(most):
                f, g = ctx[b] + kept[b, j], ctx[b] + j
                if kept[b, j] < 0 or max(f, g) >= width * page:
                    continue
                pf, pg = table[b, f // page], table[b, g // page]
                if 0 <= pf < pages and 0 <= pg < pages:
                    new[pg, :, g % page] = old[pf, :, f % page]
        assert torch.equal(t, new)


def test_refusals():
    torch = torch_cuda()
    c = cla.KVCache(8, 16, 2, 64, "int8")
    pool = cla.PagePool(8, 16, 3, 4)
    two, three = ints([0, 1]), ints([0, 1, 2])
    t, l, f = pool.block_table, pool.lens, pool.refs
    for call in (lambda: c.copy_pages(two, three), lambda: c.copy_pages(two.long(), two), lambda: c.copy_pages(two.cpu(), two.cpu()),
                 lambda: c.keep(t, l, ints([[0], [1]])), lambda: c.keep(t, l[:2], ints([[0], [1], [2]])),
                 lambda: c.keep(t[0], l, ints([[0]])), lambda: pool.extend(three, 3), lambda: pool.extend(ints([0, 1, 2, 3]), -1),
                 lambda: pool.fork(two), lambda: pool.truncate(two), lambda: pool.truncate(three.float()), lambda: pool.compact(-1),
                 lambda: cla.PagePool(0, 16, 1, 1), lambda: cla.PagePool(page_size=16, block_table=t, lens=l),
                 lambda: cla.PagePool(page_size=16, block_table=t, lens=l[:2], refs=f),
                 lambda: cla.PagePool(page_size=16, block_table=t.long(), lens=l, refs=f),
                 lambda: cla.PagePool(page_size=16, block_table=t.cpu(), lens=l.cpu(), refs=f.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pool.truncate(l), lambda: cla.PagePool(8, 17, 1, 1).fork(ints([0])), lambda: c.keep(t, l, ints(np.zeros((3, 257)))),
                 lambda: cla.PagePool(8, 16, 4097, 1).fork(ints(np.zeros(4097)))):
        with pytest.raises(cla.ClError):
            call()
    assert [x.numel() for x in pool.compact(0)] == [0, 0]
    c.keep(t, l, ints(np.zeros((3, 0))))


# ------------------------------------------------------------- used together
@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_sequences_keep_their_tokens(kind):
    """Sequences are lists of tokens; whatever is extended, forked, kept, cut and compacted, each one's entries read back as its
    tokens', in two caches that share the pool."""
    torch = torch_cuda()
    r = np.random.default_rng(11)
    pages, page, B, width, heads, dim = 120, 16, 8, 12, 2, 64
    caches = [cla.KVCache(pages, page, heads, dim, kind) for _ in range(2)]
    pool = cla.PagePool(pages, page, B, width)
    lists: list = [[] for _ in range(B)]
    number = 0

    def entries(tokens, layer):  # a token's keys: its number in base 5, in the channels
        a = np.zeros((len(tokens), heads, dim), np.float32)
        for i in range(7):
            a[:, :, 4 * i] = (np.asarray(tokens)[:, None] // 5 ** i % 5 + 1) * (layer + 1)
        return torch.from_numpy(a).cuda()

    def read_back():
        assert pool.lens.tolist() == [len(s) for s in lists]
        table = pool.block_table.cpu().numpy()
        for b, tokens in enumerate(lists):
            if not tokens:
                continue
            at = np.arange(len(tokens))
            slots = ints(table[b, at // page] * page + at % page)
            for layer, c in enumerate(caches):
                k, v = c.read(slots, dtype=torch.float32)
                want = entries(tokens, layer)
                # one code's rounding: the numbers are 1 to 5, a step at most 10 / 7
                level = (k[:, 0, ::4][:, :7] / (layer + 1)).round()
                assert torch.equal(level, want[:, 0, ::4][:, :7] / (layer + 1)) or kind == "int4"
                q, s = serving_ref.quantise(want.cpu().numpy(), kind)
                stored = torch.from_numpy(serving_ref.stored(q, s, kind).astype(np.float32)).cuda()
                assert torch.equal(k, stored) and torch.equal(v, -stored)

    for step in range(60):
        what = r.integers(5)
        say("together", kind, step, what)
        if what <= 1:  # drafts, of which some stay
            counts = [int(r.integers(0, 25)) if len(s) < 120 and r.random() < 0.7 else 0 for s in lists]
            cu = cu_of(counts)
            ctx = pool.lens.clone()
            slots, src, dst = pool.extend(ints(cu), int(cu[-1]))
            out = slots.cpu().numpy()
            new = [number + i for i in range(int(cu[-1]))]
            number += len(new)
            for layer, c in enumerate(caches):
                c.copy_pages(src, dst)
                if new:
                    e = entries(new, layer)
                    c.append(e, -e, slots)
            kept = np.full((B, 24), -1, np.int64)
            want = np.full(B, -1, np.int64)
            left = 0
            for b in range(B):
                mine = new[cu[b]:cu[b + 1]]
                if mine and out[cu[b]] < 0:
                    left += 1
                    continue
                n = int(r.integers(0, len(mine) + 1))
                path = r.permutation(len(mine))[:n]
                kept[b, :n] = path
                want[b] = len(lists[b]) + n
                lists[b] = lists[b] + [mine[i] for i in path]
            assert int(pool.left_out) == left
            for c in caches:
                c.keep(pool.block_table, ctx, ints(kept))
            pool.truncate(ints(want))
        elif what == 2:
            parents = np.where(r.random(B) < 0.4, r.integers(-1, B, B), np.arange(B))
            pool.fork(ints(parents))
            lists = [list(lists[p]) if p >= 0 else [] for p in parents]
        elif what == 3:
            cut = [int(r.integers(0, len(s) + 1)) if r.random() < 0.3 else -1 for s in lists]
            pool.truncate(ints(cut))
            lists = [s[:n] if n >= 0 else s for s, n in zip(lists, cut)]
        else:
            src, dst = pool.compact(int(r.integers(1, 40)))
            for c in caches:
                c.copy_pages(src, dst)
        read_back()


def test_step_in_a_graph():
    """A step (room, append, drafts kept, the rest taken back) recorded once and replayed: the pool moves on by itself."""
    torch = torch_cuda()
    pages, page, B, width = 200, 16, 4, 20
    r = np.random.default_rng(3)
    pool, model = cla.PagePool(pages, page, B, width), ref.Pool(pages, page, B, width)
    cache = cla.KVCache(pages, page, 2, 64, "int8")
    both(pool, model, "extend", cu_of([30, 5, 16, 1]), 52)
    cu, kept, new = cu_of([6, 6, 6, 6]), ints(np.full((B, 6), -1)), ints(np.zeros(B))
    k = torch.randn(24, 2, 64, device="cuda")
    cu_dev, ctx = ints(cu), ints(np.zeros(B))
    before = torch.zeros_like(pool.lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        before.copy_(pool.lens)
        slots, src, dst = pool.extend(cu_dev, 24)
        cache.copy_pages(src, dst)
        cache.append(k, -k, slots)
        cache.keep(pool.block_table, before, kept)
        torch.add(before, new, out=ctx)
        pool.truncate(ctx)
    same(pool, model)  # recording has run nothing
    for step in range(6):
        paths = [sorted(r.permutation(6)[:r.integers(0, 6)]) for _ in range(B)]
        list_ = np.full((B, 6), -1)
        for b, p in enumerate(paths):
            list_[b, :len(p)] = p
        kept.copy_(ints(list_))
        new.copy_(ints([len(p) for p in paths]))
        k.copy_(torch.randn(24, 2, 64, device="cuda"))
        old = model.lens.copy()
        graph.replay()
        want, s, d = model.extend(cu, 24)
        model.truncate(old + [len(p) for p in paths])
        torch.cuda.synchronize()
        assert np.array_equal(slots.cpu().numpy(), want)
        same(pool, model)
        for b, p in enumerate(paths):
            if not p:
                continue  # the reference quantises no empty lists
            at = old[b] + np.arange(len(p))
            got, _ = cache.read(ints(model.table[b, at // page] * page + at % page), dtype=torch.float32)
            q, sc = serving_ref.quantise(k[6 * b + np.array(p, int)].cpu().numpy().reshape(len(p), 2, 64), "int8")
            assert np.array_equal(got.cpu().numpy(), serving_ref.stored(q, sc, "int8").astype(np.float32))
        if step == 2:  # eager work between the replays
            both(pool, model, "fork", [0, 0, 2, 3])
