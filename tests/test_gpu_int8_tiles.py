"""The 8-bit integer product by every tile, in parts of K and in halves, bit by bit (needs an MI355X).

The sums are exact in 64-bit floats; the roundings after them are stated, so that nothing is left to a tolerance.  Which tile a size
gets is checked without a GPU.
"""
import sys

import pytest

import compressed_linear_amd as cla
import int8_bits as ref
import serving_ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def made(T, K, N, seed):
    """Codes and scales of tokens, and of a layer."""
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, w = (torch.randint(-128, 128, (n, K), dtype=torch.int8, device="cuda", generator=g) for n in (T, N))
    s = torch.rand(T, device="cuda", generator=g) * 49 + 1
    ws = (torch.rand(N, device="cuda", generator=g) * 1.5 + 0.5) / (127 * 127 * K ** 0.5)
    return q, s, w, ws, torch.randn(N, device="cuda", generator=g)


def outputs(q, s, w, ws, bias):
    """float32: an exact sum rounded, each product with a scale rounded, the sum with the bias rounded."""
    torch = torch_cuda()
    y = torch.mm(q.double(), w.double().t().contiguous()).float()
    y = y * s[:, None]
    y = y * ws
    return y if bias is None else y + bias


@pytest.mark.parametrize("T,K,N", list(ref.PLANS))
def test_every_tile(T, K, N):
    torch = torch_cuda()
    q, s, w, ws, bias = made(T, K, N, T + K)
    for b in (bias, None):
        layer = cla.Int8Linear(w, ws, bias=b)
        want = outputs(q, s, w, ws, b)
        for dst in ("f32", "f16", "bf16"):
            dt = serving_ref.torch_dtype(torch, dst)
            say("tile", T, K, N, dst, b is not None)
            room = torch.full((T + 2, N), 7.0, dtype=dt, device="cuda")
            got = layer.forward_codes(q, s, out=room[1:1 + T])
            assert torch.equal(got, want.to(dt)), int((got != want.to(dt)).sum())
            assert bool((room[0] == 7.0).all()) and bool((room[1 + T] == 7.0).all())


@pytest.mark.parametrize("T,K,N,src,dst", [(64, 8192, 28672, "bf16", "f32"), (256, 28672, 8192, "bf16", "bf16"),
                                           (777, 4099, 11005, "f32", "f16"), (2048, 8192, 28672, "bf16", "bf16")])
def test_layers_of_a_model(T, K, N, src, dst):
    torch = torch_cuda()
    _, _, w, ws, bias = made(1, K, N, T)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(T, K, device="cuda", generator=g).to(serving_ref.torch_dtype(torch, src))
    layer = cla.Int8Linear(w, ws, bias=bias, clamp=2.5)
    say("layer", T, K, N)
    got = layer(x, out_dtype=serving_ref.torch_dtype(torch, dst))
    codes, scale = cla.quantize_rows(x, clamp=2.5)  # compared bit by bit elsewhere
    assert torch.equal(got, layer.forward_codes(codes, scale, out_dtype=got.dtype))
    some = torch.unique(torch.cat([torch.arange(0, T, max(1, T // 100)), torch.tensor([T - 2, T - 1])])).cuda()
    want = outputs(codes[some], scale[some], w, ws, bias).to(got.dtype)
    assert torch.equal(got[some], want)


@pytest.mark.parametrize("K,N", list(ref.ROWS))
def test_rows_have_the_same_bits_by_any_tile(K, N):
    torch = torch_cuda()
    most = max(ref.ROWS[K, N])
    q, s, w, ws, bias = made(most, K, N, N)
    layer = cla.Int8Linear(w, ws, bias=bias)
    for dst in ("f32", "bf16", "f16"):
        dt = serving_ref.torch_dtype(torch, dst)
        whole = layer.forward_codes(q, s, out_dtype=dt)
        for T in ref.ROWS[K, N]:
            say("rows", K, N, T, dst)
            at = (most - T) // 2
            assert torch.equal(layer.forward_codes(q[at:at + T], s[at:at + T], out_dtype=dt), whole[at:at + T])


def test_tiles_in_a_graph_and_on_a_stream():
    torch = torch_cuda()
    for T, K, N in ((193, 2925, 17119), (1354, 891, 24653), (72, 18413, 1187)):
        q, s, w, ws, bias = made(T, K, N, 5)
        layer = cla.Int8Linear(w, ws, bias=bias)
        x = torch.randn(T, K, device="cuda").bfloat16()
        want = layer(x)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = layer(x)
        side.synchronize()
        assert torch.equal(got, want)
        say("graph", T, K, N)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(x)
        for _ in range(3):
            x.copy_(torch.randn(T, K, device="cuda").bfloat16())
            y.zero_()
            graph.replay()
            eager = layer(x)
            torch.cuda.synchronize()
            assert torch.equal(y, eager)
