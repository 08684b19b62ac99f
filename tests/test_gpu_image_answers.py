"""The operators of examples/image_answers.py together (needs an MI355X): against 64 bits, and answers that share a prompt's pages
against answers that have their own."""
import os
import sys

import numpy as np
import pytest

import int8_ref
import serving_ref as ref
from gpu_util import torch_cuda
from test_gpu_rope_axes import axis_of, rotate

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def linear(layer, x):
    """The layer in 64 bits from its codes, and the magnitude that rounded inputs are off by: x float16 values."""
    q, s = int8_ref.quantise(x)
    w, ws = layer.codes[:, :layer.K].cpu().numpy(), layer.scale.cpu().numpy()
    return int8_ref.product(q, s, w, ws)[0]


def start(kind="int8", n=4):
    torch = torch_cuda()
    import image_answers as ex
    a = ex.Answers(n, kind)
    g = torch.Generator(device="cuda").manual_seed(5)
    image = torch.randn(5, 7, ex.HIDDEN, generator=g, device="cuda")
    text = torch.arange(12, device="cuda") * 31 % ex.VOCAB
    return ex, a, image, text, a.prompt(text, image, text + 100)


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_prompt_against_64_bits(kind):
    torch = torch_cuda()
    import image_answers as ex
    a = ex.Answers(2, kind)
    r = np.random.default_rng(3)
    T = 30
    hidden = torch.from_numpy(r.normal(0, 1, (T, ex.HIDDEN)).astype(np.float32)).cuda()
    pos = r.integers(0, 200, (3, T))
    say("prompt", kind)
    _, logits = a.forward(hidden, [T, 0], torch.from_numpy(pos).cuda())
    x = ex.norm(hidden)
    qkv = linear(a.qkv, x.float().cpu().numpy()).reshape(T, -1, ex.DIM)
    tab, axis = a.rope.double().cpu().numpy(), axis_of(ex.SECTIONS, ex.ORDER)
    q = rotate(qkv[:, :ex.Q_HEADS], pos, axis, tab, "half").astype(np.float16).astype(np.float64)
    k = rotate(qkv[:, ex.Q_HEADS:ex.Q_HEADS + ex.KV_HEADS], pos, axis, tab, "half")
    at = torch.arange(T, device="cuda")
    slots = (a.pool.block_table[0, at // ex.PAGE] * ex.PAGE + at % ex.PAGE).to(torch.int32)
    ks, vs = (t.double().cpu().numpy() for t in a.cache.read(slots, dtype=torch.float32))
    for got, want in ((ks, k), (vs, qkv[:, ex.Q_HEADS + ex.KV_HEADS:])):
        # within half a quantisation step, the scale's own rounding and fp32's error
        width, most, clip = (ex.DIM, 127, 2.0 ** -10) if kind == "int8" else (32, 7, 2.0 ** -8)
        g = np.abs(want).reshape(T, ex.KV_HEADS, -1, width).max(-1)
        step = np.repeat(g / most, width, -1)
        assert (np.abs(got - want) <= step * (0.5 + most * clip) + 1e-4 * np.abs(want).max()).all()
    see = np.tril(np.ones((T, T), bool))
    group = ex.Q_HEADS // ex.KV_HEADS
    o = np.stack([ref.attention(q[:, i], ks[:, i // group], vs[:, i // group], see, 1 / np.sqrt(ex.DIM))[0]
                  for i in range(ex.Q_HEADS)], 1).reshape(T, -1)
    h = hidden.double().cpu().numpy() + linear(a.o, o.astype(np.float16).astype(np.float32))
    want = linear(a.head, ex.norm(torch.from_numpy(h.astype(np.float32)).cuda()).float().cpu().numpy())
    # an input that rounds the other way moves a code of o or of the head by one: a step of 1/127 of its row's largest times a weight.
    # At most a tenth of the codes do (inputs differ by 2^-10 relative, 2^-10 * 127 = 0.12 of a step), independently signed or not:
    w, ws = np.abs(a.head.codes.cpu().numpy().astype(np.float64)), a.head.scale.double().cpu().numpy()
    step = np.abs(ex.norm(torch.from_numpy(h.astype(np.float32)).cuda()).float().cpu().numpy()).max(-1) / 127
    wo, wos = np.abs(a.o.codes.cpu().numpy().astype(np.float64)), a.o.scale.double().cpu().numpy()
    moved = 0.25 * (np.abs(o).max(-1) / 127)[:, None] * (wo.sum(1) * wos)  # of h, where every fourth code of o moves
    rel = moved.max(-1) / np.sqrt((h * h).mean(-1))
    tol = (0.25 * step + rel)[:, None] * (w.sum(1) * ws) + 1e-5
    assert (np.abs(logits.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_forked_answers_are_answers_of_their_own(kind):
    torch = torch_cuda()
    ex, a, image, text, choices = start(kind)
    a.fork(4)
    assert a.pool.lens.tolist() == [59] * 4 and int((a.pool.refs > 0).sum()) == 4
    say("forked", kind, choices)
    first = [[c, 5, 6] for c in choices]
    out = a.step(first)
    for b, c in enumerate(choices):
        _, own, _, _, again = start(kind, 1)
        assert again == choices
        alone = own.step([first[b]])[0]
        # the same kernels on the same rows but for the tiles of a product: integers, so the same bits
        assert alone == out[b]
        n = int(own.pool.lens[0])
        assert n == int(a.pool.lens[b])
        at = torch.arange(n, device="cuda")
        entries = [m.cache.read((m.pool.block_table[i, at // ex.PAGE] * ex.PAGE + at % ex.PAGE).to(torch.int32)) for m, i in ((a, b), (own, 0))]
        assert all(torch.equal(x, y) for x, y in zip(*entries))


def test_answers_end_and_pages_return():
    torch = torch_cuda()
    ex, a, image, text, choices = start()
    a.fork(3)
    drafts = [[c, 1, 2, 3] for c in choices[:3]] + [[]]
    for _ in range(6):
        out = a.step(drafts)
        drafts = [[c[0], c[0], c[1], c[2]] for _, c in out[:3]] + [[]]
    lens = a.pool.lens.tolist()
    table = a.pool.block_table.clone()
    at = torch.arange(lens[2], device="cuda")
    old = a.cache.read((table[2, at // ex.PAGE] * ex.PAGE + at % ex.PAGE).to(torch.int32))
    a.end([0, 1])
    assert a.pool.lens.tolist() == [0, 0, lens[2], 0]
    held = -(-lens[2] // ex.PAGE)
    assert a.pool.refs.tolist() == [1] * held + [0] * (ex.PAGES - held)
    new = a.cache.read((a.pool.block_table[2, at // ex.PAGE] * ex.PAGE + at % ex.PAGE).to(torch.int32))
    assert all(torch.equal(x, y) for x, y in zip(old, new))
    more = a.step([[], [], [9, 9], []])  # and it goes on
    assert more[2][0][0] == 9 and int(a.pool.lens[2]) == lens[2] + len(more[2][0])
    with pytest.raises(ValueError):
        a.step([[], [], [], []])
    with pytest.raises(RuntimeError, match="pages"):
        a.forward(torch.zeros(240, ex.HIDDEN, device="cuda"), [0, 0, 240, 0], torch.zeros(3, 240, device="cuda"))
        a.forward(torch.zeros(240, ex.HIDDEN, device="cuda"), [0, 0, 240, 0], torch.zeros(3, 240, device="cuda"))
