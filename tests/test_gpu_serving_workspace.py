"""Workspaces of the attention: one to a stream, one to a recording (needs an MI355X)."""
import pytest

import compressed_linear_amd as cla
from test_gpu_serving_attention import Problem

pytestmark = pytest.mark.gpu


def test_warm_up_and_two_graphs_on_one_stream():
    # the usual recipe: an eager call on a side stream, recordings there, replays on the main stream.  By the addresses, no two
    # share a workspace, so nothing has to order them; every run here ends before the next begins.
    p = Problem([400, 33, 1200], [4, 1, 7], 8, 2, 128, 32, "int8", "bf16", seed=19)
    torch = p.torch
    want = p.call()
    tab, ctx, cu = p.dev(p.table), p.dev(p.ctx), p.dev(p.cu)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(out=None):
        return cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=p.max_q, max_ctx=1200, tree_mask=p.mask, out=out)

    with torch.cuda.stream(s):
        warm = call()
    s.synchronize()
    assert torch.equal(warm, want)
    eager = {a for a, _ in p.cache._work.values()}
    assert len(eager) == 2  # the main stream's and this one's
    graphs = []
    for _ in range(2):
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(out)
            call(out)
        graphs.append((g, out))
    recorded = {a for a, _ in p.cache._work.values()} - eager
    assert len(recorded) == 2
    for _ in range(3):
        for g, out in graphs:
            out.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        with torch.cuda.stream(s):
            again = call()
        torch.cuda.synchronize()
        assert torch.equal(again, want) and torch.equal(call(), want)


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("new,hint", [(64, 131072), (2, 2 ** 31 - 1), (33, 1000000)])
def test_chunks_that_the_workspace_limits(kind, new, hint):
    # many rows and a hint far past the real lengths: longer, fewer chunks, or one
    p = Problem([9000] + [20 * i for i in range(39)], [new] * 40, 16, 8, 64, 64, kind, "bf16", mask="tree", seed=61)
    p.check(p.call(max_ctx=hint))
    assert p.torch.equal(p.call(max_ctx=hint), p.call(max_ctx=hint))


def test_graphs_after_their_recording():
    # the cache lets a recording's workspace go; the graph keeps its memory, and a deleted graph returns it
    p = Problem([400, 33, 1200], [4, 1, 7], 8, 2, 128, 32, "int8", "bf16", seed=23)
    torch = p.torch
    want = p.call()
    tab, ctx, cu = p.dev(p.table), p.dev(p.ctx), p.dev(p.cu)
    s = torch.cuda.Stream()

    def call(out=None, max_ctx=1200):
        return cla.tree_attention(p.q, p.cache, tab, ctx, cu, max_q=p.max_q, max_ctx=max_ctx, tree_mask=p.mask, out=out)

    graphs = []
    torch.cuda.synchronize()
    for i in range(7):
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(out, max_ctx=500 * (i + 1))  # another cut of the keys
            call(out, max_ctx=4000)           # which may need a larger workspace
        graphs.append((g, out))
    assert p.cache._recorded <= 5
    assert torch.equal(call(), want) and p.cache._recorded == 0 and len(p.cache._keep) == 1
    for _ in range(3):
        for g, out in graphs:
            out.zero_()
            other = [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(10, 24)]
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            p.check(out)
            assert all(bool((t == 255).all()) for t in other)
    del other, graphs, g, out
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_reserved()
    for _ in range(12):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(max_ctx=4000)
        del g
        call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert torch.cuda.memory_reserved() <= before + (8 << 20)
