"""A pass of examples/image_answers.py that finds no room leaves every answer as it was (needs an MI355X)."""
import os
import sys

import pytest

from gpu_util import torch_cuda

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def entries(ex, a, b):
    torch = torch_cuda()
    at = torch.arange(int(a.pool.lens[b]), device="cuda")
    slots = (a.pool.block_table[b, at // ex.PAGE] * ex.PAGE + at % ex.PAGE).to(torch.int32)
    return torch.stack(a.cache.read(slots))


def start():
    torch = torch_cuda()
    import image_answers as ex
    a = ex.Answers(4)
    g = torch.Generator(device="cuda").manual_seed(5)
    image = torch.randn(5, 7, ex.HIDDEN, generator=g, device="cuda")
    text = torch.arange(12, device="cuda") * 31 % ex.VOCAB
    return ex, a, a.prompt(text, image, text + 100)


def test_answers_without_room_stay_as_they_were():
    torch = torch_cuda()
    ex, a, choices = start()
    a.fork(4)
    assert a.pool.lens.tolist() == [59] * 4  # the last page of 11 tokens is everyone's
    before = [entries(ex, a, b) for b in range(4)]
    positions = list(a.next_position)
    a.pool.refs[7:] += 1  # three free pages are left: the first three answers' copies of that page
    counts = [5, 5, 5, 30]
    say("forward", counts)
    with pytest.raises(RuntimeError, match="pages"):
        a.forward(torch.ones(45, ex.HIDDEN, device="cuda"), counts, torch.full((3, 45), 60, device="cuda"))
    assert a.pool.lens.tolist() == [59] * 4 and a.next_position == positions
    assert all(torch.equal(entries(ex, a, b), before[b]) for b in range(4))
    table, refs = a.pool.block_table.cpu(), a.pool.refs.cpu()
    assert torch.equal(torch.bincount(table[table >= 0].long(), minlength=7)[:7].int(), refs[:7])
    a.pool.refs[7:] -= 1
    # and the next pass gives what it gives where nothing had gone wrong
    drafts = [[c, 5, 6] for c in choices]
    _, other, again = start()
    other.fork(4)
    assert again == choices and a.step(drafts) == other.step(drafts)
    assert all(torch.equal(entries(ex, a, b), entries(ex, other, b)) for b in range(4))


def test_a_pass_without_room_for_one_answer_alone():
    torch = torch_cuda()
    ex, a, _ = start()
    before = entries(ex, a, 0)
    a.pool.refs[4:] += 1
    say("forward alone")
    with pytest.raises(RuntimeError, match="pages"):
        a.forward(torch.ones(12, ex.HIDDEN, device="cuda"), [5, 7, 0, 0], torch.full((3, 12), 60, device="cuda"))
    assert a.pool.lens.tolist() == [59, 0, 0, 0] and torch.equal(entries(ex, a, 0), before)
    assert int(a.pool.refs[:4].sum()) == 4 and bool((a.pool.block_table[1:] == -1).all())
