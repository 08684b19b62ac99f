"""Calls whose work is 2^32 threads and more, which no one launch holds (needs an MI355X)."""
import numpy as np
import pytest

import compressed_linear_amd as cla
import serving_ref as ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def test_rope_of_2_to_the_32_threads():
    # 17 GB of output from one token's heads
    torch = torch_cuda()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough memory")
    H, T, D = 21846, 65537, 6
    r = np.random.default_rng(3)
    one = torch.from_numpy(r.normal(0, 1, (1, H, D)).astype(np.float32)).cuda().half()
    pos = torch.from_numpy(r.integers(0, 50, T).astype(np.int32)).cuda()
    table = cla.rope_table(50, 2)
    print("rope", T, H, D, flush=True)
    y = cla.rope(one.expand(T, H, D), pos, table)
    for at in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
        assert torch.equal(y[at], cla.rope(one.expand(3, H, D), pos[at].contiguous(), table))
    del y
    torch.cuda.empty_cache()


def test_append_of_2_to_the_32_threads():
    torch = torch_cuda()
    T, H, D = (1 << 24) + 5, 16, 128
    r = np.random.default_rng(4)
    one = torch.from_numpy(r.normal(0, 1, (1, H, D)).astype(np.float32)).cuda()
    cache = cla.KVCache(2, 16, H, D, "int8")
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[0], slots[1 << 23], slots[T - 6], slots[T - 1] = 1, 4, 9, 31
    print("append", T, H, D, flush=True)
    cache.append(one.expand(T, H, D), -one.expand(T, H, D), slots)
    k, v = cache.read(torch.arange(32, dtype=torch.int32, device="cuda"), dtype=torch.float32)
    q, s = ref.quantise(one.cpu().numpy(), "int8")
    want = torch.from_numpy(ref.stored(q, s, "int8").astype(np.float32)).cuda()[0]
    for i in range(32):
        here = i in (1, 4, 9, 31)
        assert torch.equal(k[i], want if here else torch.zeros_like(want)) and torch.equal(v[i], -want if here else torch.zeros_like(want)), i


def test_log_probabilities_of_2_to_the_32_threads():
    torch = torch_cuda()
    T = (1 << 26) + 3
    x = torch.tensor([[0.5, 2.0, -1.0]], device="cuda")
    ids = (torch.arange(T, device="cuda") % 3).to(torch.int32)[:, None]
    print("log probabilities", T, flush=True)
    logp, entropy, top, top_logp = cla.token_logprobs(x.expand(T, 3), ids, top_k=1)
    first = cla.token_logprobs(x.expand(300, 3), ids[:300], top_k=1)
    assert torch.equal(logp[:300], first[0])
    assert bool((entropy == first[1][0]).all()) and bool((top == 1).all()) and bool((top_logp == first[3][0, 0]).all())
    assert bool((logp[:, 0] == first[0][:3, 0][ids[:, 0].long()]).all())


def test_table_of_2_to_the_32_pairs():
    # 34 GB
    torch = torch_cuda()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    P, rot = (1 << 26) + 3, 128
    print("table", P, rot, flush=True)
    table = cla.rope_table(P, rot)
    at = np.array([0, 1, (1 << 25) + 1, (1 << 26) - 9, 1 << 26, P - 1])
    a = at[:, None].astype(np.float64) * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    got = table[torch.from_numpy(at).cuda()].double().cpu().numpy()
    # one rounding to fp32, and a few fp64 roundings of an angle of up to P
    assert (np.abs(got - np.stack([np.cos(a), np.sin(a)], -1)) <= 2.0 ** -24 + 64 * P * 2.0 ** -52).all()
    del table
    torch.cuda.empty_cache()
