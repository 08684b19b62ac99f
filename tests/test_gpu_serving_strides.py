"""Queries of the attention wherever they lie in memory (needs an MI355X)."""
import pytest

from gpu_util import torch_cuda
from test_gpu_serving_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_queries_at_any_address_and_stride(dtype):
    # contiguous, but no multiple of 16 bytes; and sizes of one, whose strides mean nothing
    torch = torch_cuda()
    for new, hq, hkv in (([6, 2], 6, 2), ([1], 6, 2), ([1], 1, 1)):
        p = Problem([130, 9][:len(new)], new, hq, hkv, 128, 16, "int8", dtype, seed=2)
        want = p.call()
        T = int(p.new.sum())
        for lead in (1, 3, 4):
            room = torch.zeros(p.q.numel() + 8, dtype=p.q.dtype, device="cuda")
            q = room[lead:lead + p.q.numel()].view(p.q.shape)
            q.copy_(p.q)
            assert q.is_contiguous() and torch.equal(p.call(q=q), want)
        if T == 1:
            room = torch.zeros(p.q.numel() + 8, dtype=p.q.dtype, device="cuda")
            head = 128 if hq > 1 else 131
            q = room.as_strided(p.q.shape, (hq * 128 + 5, head, 1))
            q.copy_(p.q)
            assert torch.equal(p.call(q=q), want)
