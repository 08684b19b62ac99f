"""Log probabilities of logits of any size against 64 bits (needs an MI355X).

The bound follows from what is rounded, before any run: x - m is one fp32 rounding of the difference, so that the logits' own
size does not enter.  With d = x - m, p the probabilities, W = sum p |d| and W2 = sum p d^2: a term of l = sum e^d is off
by its exponent's two roundings and exp2's (2^-24 (4 |d| + 4) of itself), the sum by at most V / 64 + 64 roundings; log l by 4 2^-24 of
itself besides; w = sum d e^d alike, each term weighted with |d|.
"""
import numpy as np
import pytest

import compressed_linear_amd as cla
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("V", [300, 3000, 40003])
def test_large_logits(V):
    torch = torch_cuda()
    r = np.random.default_rng(V)
    x = np.stack([np.full(V, -3e38), np.full(V, 3e38), r.normal(0, 1, V) * 1e30, r.normal(0, 1, V) + 1e4, r.normal(0, 1, V) - 3e6,
                  r.normal(0, 100, V), np.r_[3.0, np.full(V - 1, -3e38)]]).astype(np.float32)
    ids = np.stack([np.zeros(7, int), np.full(7, V - 1), r.integers(0, V, 7)], 1).astype(np.int32)
    logp, ent, top, toplp = (t.double().cpu().numpy() for t in cla.token_logprobs(torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), top_k=12))
    d = x.astype(np.float64)
    d -= d.max(-1, keepdims=True)
    e = np.exp(d)
    l = e.sum(-1, keepdims=True)
    p, lse = e / l, np.log(l)
    with np.errstate(over="ignore", invalid="ignore"):
        W, W2 = (np.where(p > 0, p * np.abs(d) ** n, 0).sum(-1) for n in (1, 2))
    want = (lse[:, 0] + W, d - lse)
    order = np.stack([np.lexsort((np.arange(V), -x[t])) for t in range(7)])[:, :12]
    assert np.array_equal(top, order)
    sums = 4 * W + V / 64 + 80  # of l, relative

    def check(got, at):
        w, a = np.take_along_axis(want[1], at, 1), np.take_along_axis(np.abs(d), at, 1)
        tol = U * (2 * a + sums[:, None] + 4 * np.abs(lse) + 2 * np.abs(w))
        assert np.isfinite(tol).all() and (np.abs(got - w) <= tol).all(), np.abs(got - w) / tol
    check(logp, ids.astype(np.int64))
    check(toplp, order)
    tol = U * (4 * W2 + W * (V / 64 + 80 + sums) + sums + 4 * np.abs(lse[:, 0]) + 2 * np.abs(want[0]))
    assert np.isfinite(tol).all() and (np.abs(ent - want[0]) <= tol).all(), np.abs(ent - want[0]) / tol
    assert ent[2] == 0 and ent[6] == 0 and (tol[:2] < 1e-4).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("V", [70, 3000, 40003])
def test_rows_masked_with_the_lowest_value(V, dtype):
    # a constrained row: few logits left, the others the type's lowest value (or a mix of it and -inf)
    torch = torch_cuda()
    dt = getattr(torch, dtype)
    low = torch.finfo(dt).min
    r = np.random.default_rng(V + 1)
    x = torch.full((6, V), low, dtype=dt, device="cuda")
    left = [[V - 1], [0, V // 2], [5], list(range(40)), [], r.permutation(V)[:9].tolist()]
    for t, at in enumerate(left):
        x[t, at] = torch.from_numpy(r.normal(0, 3, len(at)).astype(np.float32)).cuda().to(dt)
    x[2, V // 3:] = -float("inf")
    logp, ent, top, _ = cla.token_logprobs(x, torch.tensor([[5, V - 1]] * 6, dtype=torch.int32, device="cuda"), top_k=8)
    d = x.double()
    want = torch.log_softmax(d, -1)
    p = want.exp()
    h = -torch.where(p > 0, p * want, 0).sum(-1)
    # as above with |d| below 20 (or p = 0) and entropies below log V
    assert bool(((ent - h).abs() <= U * (4 * 400 + 20 * (V / 32 + 240) + V / 64 + 200)).all()), (ent, h)
    w = want[:, [5, V - 1]]
    fine = w > -1e30
    assert bool(((logp - w).abs() <= U * (4 * w.abs() + 4 * 20 + V / 64 + 200))[fine].all()) and not bool(logp.isnan().any())
    assert torch.equal(top.long(), torch.sort(d, dim=-1, descending=True, stable=True).indices[:, :8])
