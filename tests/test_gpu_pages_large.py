"""Operations on the pages of a cache whose tables are wider than a launch is (needs an MI355X)."""
import sys

import pytest

import compressed_linear_amd as cla
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def test_fork_of_a_table_wider_than_a_launch():
    # 16 columns to a workgroup of 1024: 2^26 columns are 2^32 threads (1.1 GB of table, counts and copies)
    torch = torch_cuda()
    width, page = (1 << 26) + 40, 16
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(width, dtype=torch.int32, device="cuda")
    lens = torch.tensor([width * page - 3, 0], dtype=torch.int32, device="cuda")
    refs = torch.zeros(width + 5, dtype=torch.int32, device="cuda")
    refs[:width] = 1
    pool = cla.PagePool(page_size=page, block_table=table, lens=lens, refs=refs)
    row = table[0].clone()
    say("fork", width)
    pool.fork(torch.tensor([0, 0], dtype=torch.int32, device="cuda"))
    assert lens.tolist() == [width * page - 3] * 2
    assert torch.equal(table[0], row) and torch.equal(table[1], row)
    assert bool((refs[:width] == 2).all()) and not refs[width:].any()
    say("end and trade places")
    pool.fork(torch.tensor([-1, 0], dtype=torch.int32, device="cuda"))
    assert lens.tolist() == [0, width * page - 3]
    assert bool((table[0] == -1).all()) and torch.equal(table[1], row)
    assert bool((refs[:width] == 1).all())
    pool.fork(torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    assert lens.tolist() == [width * page - 3, 0] and torch.equal(table[0], row) and bool((table[1] == -1).all())
    assert bool((refs[:width] == 1).all())
