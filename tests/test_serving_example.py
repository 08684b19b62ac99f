"""The parts of the example of the serving operators that need no GPU."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_trees_of_up_to_64_drafts():
    import verify_drafts as ex
    for T in (1, 6, 63, 64):
        parents = [-1, -1] + [i // 2 for i in range(T - 2)] if T > 2 else [-1] * T
        mask, depth = ex.tree_of(parents)
        assert mask.shape == (T, 1) and mask.dtype == torch.int64 and depth.dtype == torch.int64
        for i in range(T):
            up, n = {i}, 0
            at = parents[i]
            while at >= 0:
                up.add(at)
                at, n = parents[at], n + 1
            assert {j for j in range(64) if (int(mask[i, 0]) >> j) & 1} == up and int(depth[i]) == n


def test_more_tokens_than_the_pages_hold_are_refused():
    import verify_drafts as ex
    most = ex.PAGE * ex.PAGES
    for n, new in ((0, 1), (0, ex.MAX_NEW), (most - 5, 5)):
        ex.room(n, new)
    for n, new in ((most, 1), (most - 5, 6), (0, ex.MAX_NEW + 1), (3, 0)):
        with pytest.raises(ValueError):
            ex.room(n, new)
    block = object.__new__(ex.Block)  # refused before anything is done
    block.n, block.embed = most - 1, torch.zeros(2, 2)
    with pytest.raises(ValueError, match="pages"):
        block.forward(torch.tensor([0, 1]), torch.tensor([0, 1]))
    with pytest.raises(ValueError, match="empty"):
        block.prompt(torch.tensor([], dtype=torch.int64))
