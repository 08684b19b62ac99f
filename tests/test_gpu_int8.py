"""The linear layer in 8-bit integers against plain references (needs an MI355X).

Codes and scales are defined down to each fp32 rounding and compared bit by bit; sums of integers are exact, so that the
outputs are off by the roundings after them only.
"""
import sys

import numpy as np
import pytest

import compressed_linear_amd as cla
import int8_ref as ref
import serving_ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def values(r, shape, dtype):
    torch = torch_cuda()
    return torch.from_numpy(r.normal(0, 1, shape).astype(np.float32)).cuda().to(serving_ref.torch_dtype(torch, dtype))


def check(y, q, s, w, ws, bias, dtype):
    want, p = ref.product(q, s, w, ws, bias)
    got = y.double().cpu().numpy()
    assert got.shape == want.shape
    tol = ref.tolerance(want, p, bias, dtype)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 4096), (3, 5), (2, 127), (5, 129), (37, 1000), (300, 384), (2, 28672), (9, 10241), (3, 40001), (1, 131071)])
def test_codes(T, K, dtype):
    torch = torch_cuda()
    r = np.random.default_rng(K * 10 + T)
    x = values(r, (T, K + 7), dtype)
    for at, clamp in ((0, None), (3, 0.7)):  # 16-byte aligned rows or not
        v = x[:, at:at + K]
        say("codes", T, K, dtype, at)
        codes, scale = cla.quantize_rows(v, clamp=clamp)
        q, s = ref.quantise(v.float().cpu().numpy(), clamp or 0.0)
        assert codes.shape == (T, K) and np.array_equal(codes.cpu().numpy(), q)
        assert np.array_equal(scale.cpu().numpy(), s)
        width = -(-K // 128) * 128
        whole = torch.as_strided(codes, (T, width), (width, 1))
        assert codes.stride(0) == width and not whole[:, K:].any()


def test_rows_without_numbers():
    torch = torch_cuda()
    x = np.zeros((8, 200), np.float32)
    x[1, 3] = np.nan
    x[2, 199] = np.inf
    x[3, 0] = -np.inf
    x[4] = 2.0 ** -101
    x[5, 7] = -2.0 ** -100
    x[6] = 3e38
    x[7, 9], x[7, 10] = np.inf, 1.0
    for clamp in (None, 5.0):
        codes, scale = cla.quantize_rows(torch.from_numpy(x).cuda(), clamp=clamp)
        q, s = ref.quantise(x, clamp or 0.0)
        assert np.array_equal(codes.cpu().numpy(), q)
        assert np.array_equal(scale.cpu().numpy(), s, equal_nan=True)
        assert np.isnan(s[1]) and np.isnan(s[2]) == (clamp is None) and s[4] == 0 and s[5] > 0
        layer = cla.Int8Linear(torch.ones(5, 200, dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"), clamp=clamp)
        y = layer(torch.from_numpy(x).cuda()).cpu().numpy()
        assert np.array_equal(np.isnan(y), np.repeat(np.isnan(s)[:, None], 5, 1)) and (y[[0, 4]] == 0).all()


SIZES = [  # T, K, N
    (1, 128, 256), (1, 1, 1), (1, 1000, 77), (1, 8192, 1280), (2, 4096, 512), (3, 129, 65), (4, 2048, 300), (7, 640, 1000),
    (8, 28672, 64), (9, 256, 4096), (16, 1024, 130), (17, 300, 33), (31, 4100, 200), (32, 512, 512), (33, 513, 513),
    (48, 1280, 96), (63, 384, 2000), (64, 2048, 256), (65, 128, 129), (96, 1000, 320), (127, 900, 250), (128, 4096, 384),
    (129, 256, 260), (200, 3000, 100), (255, 130, 255), (256, 1024, 512), (257, 640, 511), (300, 129, 1025), (500, 5000, 40),
    (777, 384, 1300), (1024, 256, 1024), (1030, 1152, 770), (2048, 512, 768), (5000, 100, 20), (2049, 200, 2050),
]


@pytest.mark.parametrize("T,K,N", SIZES)
def test_product(T, K, N):
    torch = torch_cuda()
    r = np.random.default_rng(T * 7 + K * 3 + N)
    w = r.integers(-127, 128, (N, K)).astype(np.int8)
    ws = r.uniform(0.5, 2, N).astype(np.float32) * np.float32(1e-3)
    bias = r.normal(0, 1, N).astype(np.float32)
    plain = cla.Int8Linear(torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    other = cla.Int8Linear(torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda(), bias=torch.from_numpy(bias).cuda(), clamp=1.5)
    for src, dst in (("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")):
        x = values(r, (T, K), src)
        dt = serving_ref.torch_dtype(torch, dst)
        xf = x.float().cpu().numpy()
        say("product", T, K, N, src, dst)
        q, s = ref.quantise(xf)
        y = plain(x, out_dtype=dt)
        check(y, q, s, w, ws, None, dst)
        codes, scale = cla.quantize_rows(x)
        assert torch.equal(plain.forward_codes(codes, scale, out_dtype=dt), y)
        q, s = ref.quantise(xf, 1.5)
        check(other(x, out_dtype=dt), q, s, w, ws, bias, dst)


@pytest.mark.parametrize("T,K,N", [(1, 1000, 300), (5, 384, 257), (40, 130, 140), (130, 700, 300), (300, 256, 600)])
def test_strides_and_outputs(T, K, N):
    torch = torch_cuda()
    r = np.random.default_rng(T)
    w = r.integers(-127, 128, (N, K)).astype(np.int8)
    ws = r.uniform(0.5, 2, N).astype(np.float32)
    layer = cla.Int8Linear(torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    wide = values(r, (T, K + 9), "f16")
    for v in (wide[:, :K], wide[:, 5:5 + K], wide[:1, :K].expand(T, K), wide.t().contiguous().t()[:, 1:1 + K]):
        q, s = ref.quantise(v.float().cpu().numpy())
        say("strides", T, K, N, v.stride())
        check(layer(v), q, s, w, ws, None, "f32")
    q, s = ref.quantise(wide[:, :K].float().cpu().numpy())
    for dst in ("f32", "f16", "bf16"):
        dt = serving_ref.torch_dtype(torch, dst)
        for first, extra in ((0, 0), (8, 8), (3, 6)):  # aligned rows, a view of wider ones, odd addresses
            room = torch.full((T + 2, N + extra), 7.0, dtype=dt, device="cuda")
            out = room[1:1 + T, first:first + N] if extra else room[1:1 + T]
            assert layer(wide[:, :K], out=out) is out
            check(out, q, s, w, ws, None, dst)
            room[1:1 + T, first:first + N] = 7.0
            assert (room == 7.0).all()
    # rows of codes that lie apart, or whose tail is someone else's
    codes, scale = cla.quantize_rows(wide[:, :K])
    y = layer.forward_codes(codes, scale)
    assert torch.equal(layer.forward_codes(codes.contiguous(), scale), y)
    apart = torch.full((T, 256 * (K // 256 + 2)), 99, dtype=torch.int8, device="cuda")
    apart[:, :K] = codes
    assert torch.equal(layer.forward_codes(apart[:, :K], scale), y)
    apart[:, 1:K + 1] = codes
    assert torch.equal(layer.forward_codes(apart[:, 1:K + 1], scale), y)


def test_weights():
    torch = torch_cuda()
    r = np.random.default_rng(2)
    W = values(r, (70, 300), "bf16")
    x = values(r, (11, 300), "f16")
    layer = cla.Int8Linear.from_weight(W, bias=torch.arange(70, device="cuda").float())
    w, ws = ref.quantise(W.float().cpu().numpy())
    q, s = ref.quantise(x.float().cpu().numpy())
    check(layer(x), q, s, w, ws, np.arange(70, dtype=np.float32), "f32")
    assert layer(x[:0]).shape == (0, 70) and layer(x[0]).shape == (1, 70)
    assert torch.equal(layer(x[3]), layer(x)[3:4])
    # all 256 codes, the largest sums
    K = 131071
    w = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    layer = cla.Int8Linear(w, torch.ones(3, device="cuda"))
    for T in (1, 5, 40, 300):
        codes = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
        y = layer.forward_codes(codes, torch.ones(T, device="cuda"))
        assert (y == float(np.float32(128 * 128 * K))).all()
        codes[0] = 127
        assert (layer.forward_codes(codes, torch.ones(T, device="cuda"))[0] == float(np.float32(-128 * 127 * K))).all()
    assert cla.Int8Linear(w[:, :128], torch.ones(3, device="cuda")).codes.shape == (3, 128)


def test_rows_do_not_depend_on_others():
    torch = torch_cuda()
    r = np.random.default_rng(8)
    layer = cla.Int8Linear.from_weight(values(r, (384, 1500), "f32"))
    x = values(r, (700, 1500), "bf16")
    whole = layer(x)
    for T in (1, 2, 6, 20, 33, 70, 140, 300):
        say("rows", T)
        assert torch.equal(layer(x[100:100 + T]), whole[100:100 + T])
    x[5] = float("nan")
    again = layer(x)
    assert torch.isnan(again[5]).all() and torch.equal(again[6:], whole[6:])


def test_stream_and_graph():
    torch = torch_cuda()
    r = np.random.default_rng(5)
    layer = cla.Int8Linear.from_weight(values(r, (512, 640), "f32"))
    for T in (1, 12, 100, 600):
        x = values(r, (T, 640), "bf16")
        want = layer(x)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = layer(x)
        side.synchronize()
        assert torch.equal(got, want)
        say("graph", T)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(x)
        for k in range(4):
            x.copy_(values(r, (T, 640), "bf16"))
            y.zero_()
            graph.replay()
            eager = layer(x)
            torch.cuda.synchronize()
            assert torch.equal(y, eager), k


def test_more_tiles_than_a_launch_holds():
    # 137 GB of outputs: two pieces of tokens, the second of 20
    torch = torch_cuda()
    N, K, T = 1 << 23, 128, 8192 + 20
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("not enough memory")
    r = np.random.default_rng(1)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    ws = torch.rand(N, device="cuda")
    layer = cla.Int8Linear(w, ws)
    x = values(r, (T, K), "f16")
    say("pieces", T, K, N)
    y = layer(x, out_dtype=torch.float16)
    q, s = ref.quantise(x.float().cpu().numpy())
    for t in (slice(0, 3), slice(8190, 8195), slice(T - 3, T)):
        for n in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(N - 300, N)):
            check(y[t, n], q[t], s[t], w[n].cpu().numpy(), ws[n].cpu().numpy(), None, "f16")
    del y
    torch.cuda.empty_cache()


def test_refusals():
    torch = torch_cuda()
    dev = "cuda"
    codes, scale = torch.zeros(8, 64, dtype=torch.int8, device=dev), torch.ones(8, device=dev)
    layer = cla.Int8Linear(codes, scale)
    x = torch.zeros(3, 64, device=dev)
    for call in (lambda: cla.Int8Linear(codes.float(), scale), lambda: cla.Int8Linear(codes.cpu(), scale),
                 lambda: cla.Int8Linear(codes, scale[:4]), lambda: cla.Int8Linear(codes, scale.half()),
                 lambda: cla.Int8Linear(codes, scale, bias=scale.double()), lambda: cla.Int8Linear(codes, scale, clamp=-1.0),
                 lambda: cla.Int8Linear(codes, scale, clamp=0.0), lambda: cla.Int8Linear(codes, scale, clamp=float("nan")),
                 lambda: cla.Int8Linear(torch.zeros(1, 131072, dtype=torch.int8, device=dev), scale[:1]),
                 lambda: cla.Int8Linear(codes[:0], scale[:0]),
                 lambda: layer(x[:, :63]), lambda: layer(x.double()), lambda: layer(x.cpu()), lambda: layer(x[None]),
                 lambda: layer(x, out=torch.zeros(3, 7, device=dev)), lambda: layer(x, out_dtype=torch.int32),
                 lambda: layer(x, out=torch.zeros(3, 8, device=dev), out_dtype=torch.float16),
                 lambda: layer(x, out=torch.zeros(8, 3, device=dev).t()), lambda: layer(x, out=torch.zeros(1, 8, device=dev).expand(3, 8)),
                 lambda: layer.forward_codes(x, scale[:3]), lambda: layer.forward_codes(codes[:3], scale),
                 lambda: cla.quantize_rows(x.double()), lambda: cla.quantize_rows(x[:, :0]),
                 lambda: cla.quantize_rows(torch.zeros(1, 131072, device=dev)), lambda: cla.quantize_rows(x, clamp=0.0)):
        with pytest.raises(ValueError):
            call()
    assert cla.quantize_rows(x[:0])[0].shape == (0, 64)
    assert layer.forward_codes(codes[:0], scale[:0]).shape == (0, 8)


@pytest.mark.parametrize("clamp", [2.0 ** -101, 1e-45, 1e-50])
def test_clamps_below_the_least_scale_leave_zeros(clamp):
    """Every value is clamped below 2^-100, so codes and scales are zeros and a layer's outputs are its bias."""
    torch = torch_cuda()
    x = torch.linspace(-3, 3, 5 * 130, device="cuda").reshape(5, 130)
    codes, scale = cla.quantize_rows(x, clamp=clamp)
    assert not codes.any() and not scale.any()
    bias = torch.arange(7, dtype=torch.float32, device="cuda")
    layer = cla.Int8Linear.from_weight(torch.ones(7, 130, device="cuda"), bias=bias, clamp=clamp)
    assert torch.equal(layer(x), bias.expand(5, 7))
