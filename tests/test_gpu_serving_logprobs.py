"""Log probabilities of given tokens, entropy and alternatives against 64 bits (needs an MI355X).

Tolerances follow from the roundings (serving_ref.logprob_tolerance), before any run; ids have to be equal.
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


def check(xd, ids, k):
    torch = torch_cuda()
    x = xd.float().cpu().numpy()
    got = cla.token_logprobs(xd, torch.from_numpy(ids.astype(np.int32)).cuda(), top_k=k)
    logp, ent = (t.cpu().numpy() for t in got[:2])
    wlogp, went, wtop, wtopl, W = ref.logprobs(x, ids, k)
    tol = ref.logprob_tolerance(x, np.where(np.isfinite(wlogp), wlogp, 0))

    def near(a, b, t):
        fine = np.isfinite(b)
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~fine & ~np.isnan(b)], b[~fine & ~np.isnan(b)])
        assert (np.abs(a - b)[fine] <= np.broadcast_to(t, b.shape)[fine]).all(), np.abs(a - b)[fine].max()

    near(logp, wlogp, tol)
    base = ref.logprob_tolerance(x, np.zeros(1))
    near(ent, went, 2 * base * (2 + np.where(np.isfinite(W), W, 0)))
    if k:
        assert np.array_equal(got[2].cpu().numpy(), wtop)
        near(got[3].cpu().numpy(), wtopl, ref.logprob_tolerance(x, np.where(np.isfinite(wtopl), wtopl, 0)))


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,C,k", [(1, 1, 1, 1), (1, 2, 1, 2), (3, 31, 2, 31), (2, 64, 1, 32), (5, 65, 3, 5), (1, 32000, 1, 8),
                                     (7, 1023, 0, 7), (2, 50257, 4, 20), (300, 777, 1, 0), (1, 151937, 2, 32),
                                     (600, 4099, 2, 1), (33, 16384, 1, 16), (520, 9001, 1, 5), (300, 20011, 2, 32),
                                     (260, 66001, 1, 3), (9, 8195, 1, 17), (400, 1999, 2, 32),
                                     (257, 4095, 1, 20)])
def test_rows(src, T, V, C, k):
    torch = torch_cuda()
    say("logprobs", src, T, V, C, k)
    r = np.random.default_rng(T + V)
    x = r.normal(0, 2.5, (T, V))
    x[np.arange(T), r.integers(0, V, T)] += 9
    xd = torch.from_numpy(x.astype(np.float32)).cuda().to(ref.torch_dtype(torch, src))
    check(xd, r.integers(0, V, (T, C)), k)


@pytest.mark.parametrize("V", [70, 5000, 40001])
def test_ties_go_to_the_lowest_id(V):
    torch = torch_cuda()
    say("ties", V)
    r = np.random.default_rng(V)
    rows = [np.zeros(V), np.full(V, -3.5), r.integers(-2, 3, V), np.where(r.random(V) < 0.5, 0.0, -0.0),
            np.sort(r.normal(0, 1, V)), -np.sort(r.normal(0, 1, V)), np.r_[np.zeros(V - 1), 1.0], r.integers(0, 2, V) * 5.0]
    xd = torch.from_numpy(np.array(rows, np.float32)).cuda()
    for k in (1, 4, 32):
        check(xd, np.zeros((len(rows), 1), np.int64), k)


def test_infinities_nan_and_large_values():
    torch = torch_cuda()
    V = 3000
    r = np.random.default_rng(1)
    x = r.normal(0, 1, (9, V)).astype(np.float32)
    x[0, 1:] = -np.inf                # one token left
    x[1, :] = -np.inf                 # none
    x[2, 7] = np.nan
    x[3, 9] = np.inf
    x[4] = np.where(r.random(V) < 0.9, -np.inf, x[4])
    x[5] *= 1e30
    x[6] = -3e38
    x[7, 5:] = -np.inf                # fewer than top_k finite
    x[8, [3, 2999]] = np.nan
    ids = np.stack([np.zeros(9, int), np.full(9, 7), np.full(9, 9), np.full(9, V - 1), np.full(9, V), np.full(9, -1),
                    np.full(9, 2 ** 31 - 1), np.full(9, -2 ** 31)], 1)
    xd = torch.from_numpy(x).cuda()
    for i in range(9):  # each row by itself: its magnitude sets its tolerance
        say("row", i)
        check(xd[i:i + 1], ids[i:i + 1], 12)
    check(xd[:0], ids[:0], 0)


def test_strided_rows_streams_and_graph():
    torch = torch_cuda()
    r = np.random.default_rng(2)
    big = torch.from_numpy(r.normal(0, 2, (6, 5003)).astype(np.float32)).cuda()
    for dt in ("f32", "bf16"):
        wide = big.to(ref.torch_dtype(torch, dt))
        check(wide[:, 1:4000], r.integers(0, 3999, (6, 2)), 5)
        check(wide[::2, 3:], r.integers(0, 5000, (3, 2)), 5)
        check(wide.t()[:900].contiguous().t()[:, :900], r.integers(0, 900, (6, 2)), 5)  # vocabulary not contiguous
    ids = torch.zeros(6, 1, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in cla.token_logprobs(big, ids, top_k=4)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = cla.token_logprobs(big, ids, top_k=4)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = big.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = cla.token_logprobs(x, ids, top_k=4)
    for i in range(4):
        x.copy_(big * (0.5 + i))
        eager = cla.token_logprobs(x, ids, top_k=4)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i


def test_refusals():
    torch = torch_cuda()
    x = torch.zeros(3, 50, device="cuda")
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    for bad in (lambda: cla.token_logprobs(x.double(), ids), lambda: cla.token_logprobs(x[0], ids),
                lambda: cla.token_logprobs(x, ids.long()), lambda: cla.token_logprobs(x, ids[:2]),
                lambda: cla.token_logprobs(x, ids.cpu()), lambda: cla.token_logprobs(x.cpu(), ids)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cla.token_logprobs(x, ids, top_k=33), lambda: cla.token_logprobs(x[:, :4], ids, top_k=5),
                lambda: cla.token_logprobs(x, ids, top_k=-1)):
        with pytest.raises((cla.ClError, RuntimeError)):
            bad()
