"""The serving operators together with compressed layers: the example's drafted-token step (needs an MI355X).

The step is recomputed in 64 bits from the layers' dequantised weights and the cache's own entries; verifying a
chain in one pass has to say what token-by-token decoding says.
"""
import os
import sys

import numpy as np
import pytest

import compressed_linear_amd as cla
import serving_ref as ref
from gpu_util import torch_cuda

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def weights(mod):
    D16, S16, _, _ = mod.debug_dequant()
    return D16.double() + S16.double()


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_tree_step_against_64_bits(kind):
    torch = torch_cuda()
    import verify_drafts as ex
    b = ex.Block(kind)
    b.prompt(torch.arange(70, device="cuda") * 13 % ex.VOCAB)
    n = b.n
    assert n == 70
    parents = [-1, 0, 0, 2, -1, 4, 5]
    tokens = torch.tensor([5, 6, 7, 8, 9, 10, 11], device="cuda")
    T = len(tokens)
    see = np.zeros((T, T), bool)
    depth = np.zeros(T, np.int64)
    for i, p in enumerate(parents):
        if p >= 0:
            see[i] = see[p]
            depth[i] = depth[p] + 1
        see[i, i] = True
    mask = torch.tensor([[int(sum(1 << j for j in range(T) if see[i, j]))] for i in range(T)], device="cuda")
    say("tree step", kind)
    logits = b.forward(tokens, torch.from_numpy(depth).cuda(), mask)
    # the block in 64 bits, rounding where the program rounds to fp16 (its inputs to layers, q, o)
    h = b.embed[tokens]
    x = ex.norm(h).double()
    qkv = (x @ weights(b.qkv).T).view(T, -1, ex.DIM).cpu().numpy()
    tab = b.rope.double().cpu().numpy()
    q = ref.rotate(qkv[:, :ex.Q_HEADS], n + depth, tab, "half").astype(np.float16).astype(np.float64)
    every = b.slots(torch.arange(n + T, device="cuda"))
    ks, vs = (t.double().cpu().numpy() for t in b.cache.read(every, dtype=torch.float32))
    # what was appended, within half a quantisation step and fp32's error
    for got, want in ((ks[n:], ref.rotate(qkv[:, ex.Q_HEADS:ex.Q_HEADS + ex.KV_HEADS], n + depth, tab, "half")),
                      (vs[n:], qkv[:, ex.Q_HEADS + ex.KV_HEADS:])):
        width, most, clip = (ex.DIM, 127, 2.0 ** -10) if kind == "int8" else (32, 7, 2.0 ** -8)
        g = np.abs(want).reshape(T, ex.KV_HEADS, -1, width).max(-1)
        step = np.repeat(g / most, width, -1)
        assert (np.abs(got - want) <= step * (0.5 + most * clip) + 1e-4 * np.abs(want).max()).all()
    full = np.concatenate([np.ones((T, n), bool), see], 1)
    o = np.stack([ref.attention(q[:, i], ks[:, i // 4], vs[:, i // 4], full, 1 / np.sqrt(ex.DIM))[0]
                  for i in range(ex.Q_HEADS)], 1)
    o = torch.from_numpy(o.astype(np.float16)).cuda().double().view(T, -1)
    h2 = h.double() + o @ weights(b.o).T
    want = ex.norm(h2.float()).double() @ weights(b.head).T
    # fp16 inputs that round the other way here and there move a logit by 2^-11 of sum |x w| at most, twice
    tol = 2.0 ** -10 * (ex.norm(h2.float()).double().abs() @ weights(b.head).T.abs())
    assert ((logits.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_chain_in_one_pass_is_token_by_token(kind):
    torch = torch_cuda()
    import verify_drafts as ex
    prompt = torch.arange(33, device="cuda") * 7 % ex.VOCAB
    tokens = torch.tensor([1, 2, 3, 500, 999], device="cuda")
    one, many = ex.Block(kind), ex.Block(kind)
    for b in (one, many):
        b.prompt(prompt)
    mask = torch.tensor([[(1 << (i + 1)) - 1] for i in range(5)], device="cuda")
    at_once = one.forward(tokens, torch.arange(5, device="cuda"), mask)
    rows = []
    for i in range(5):
        rows.append(many.forward(tokens[i:i + 1], torch.zeros(1, dtype=torch.int64, device="cuda")))
        many.n += 1
    say("chain", kind)
    spread = at_once.abs().max()
    # layers run other kernels for one row than for five: fp32 sums in another order, then fp16 roundings
    assert (torch.cat(rows) - at_once).abs().max() <= 2.0 ** -8 * spread


def test_example_runs_and_accepts():
    torch = torch_cuda()
    import verify_drafts as ex
    b = ex.Block()
    choices = b.prompt(torch.arange(40, device="cuda")).tolist()
    b.expected = choices[0]
    n = b.n
    path, following, logp, entropy = b.verify(torch.tensor([choices[0], choices[1], 9], device="cuda"), [-1, -1, 0])
    assert path[0] == 0 and b.n == n + len(path)
    assert torch.isfinite(entropy).all() and (entropy >= 0).all()
    assert torch.isfinite(logp[0, 0]) and torch.isnan(logp[0, 1:]).all()  # one child, then padding
    # decoding the accepted token alone gives the same next choice
    again = ex.Block()
    again.prompt(torch.arange(40, device="cuda"))
    first = again.forward(torch.tensor([choices[0]], device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert int(first.argmax()) == (9 if len(path) > 1 else following)
