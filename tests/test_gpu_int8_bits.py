"""The 8-bit integer layer's outputs bit by bit, biases among them (needs an MI355X)."""
import sys

import numpy as np
import pytest

import compressed_linear_amd as cla
import int8_bits as ref
import serving_ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def compare(layer, codes, scale, want, dtypes=("f32", "f16", "bf16")):
    torch = torch_cuda()
    want = torch.from_numpy(want).cuda()
    for name in dtypes:
        dt = serving_ref.torch_dtype(torch, name)
        got = layer.forward_codes(codes, scale, out_dtype=dt)
        assert torch.equal(got, want.to(dt)), (name, int((got != want.to(dt)).sum()))


@pytest.mark.parametrize("T,K,N", [(1, 1000, 300), (7, 130, 77), (16, 640, 200), (30, 2000, 90), (64, 129, 400),
                                   (65, 300, 129), (200, 700, 333), (300, 6000, 60)])
def test_bias_is_added_to_rounded_products(T, K, N):
    torch = torch_cuda()
    r = np.random.default_rng(T + K)
    w, ws, bias = ref.weights(r, N, K)
    q, s = ref.activations(r, T, K)
    acc = ref.sums(q, w)
    codes, scale = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    say("bits", T, K, N)
    for b in (bias, None):
        layer = cla.Int8Linear(torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda(), bias=None if b is None else torch.from_numpy(b).cuda())
        compare(layer, codes, scale, ref.outputs(acc, s, ws, b))
