"""Copies of a layer in 8-bit integers do not need the layer they were made from (needs an MI355X)."""
import copy
import io
import pickle
import sys

import pytest

import compressed_linear_amd as cla
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def saved(layer):
    torch = torch_cuda()
    f = io.BytesIO()
    torch.save(layer, f)
    f.seek(0)
    return torch.load(f, weights_only=False)  # written above


@pytest.mark.parametrize("K,bias,clamp", [(128, False, None), (300, True, 1.5)])
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x)), saved],
                         ids=["copy", "deepcopy", "pickle", "save"])
def test_copies(how, K, bias, clamp):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(70, K, generator=g, device="cuda")
    layer = cla.Int8Linear.from_weight(W, bias=torch.arange(70, device="cuda").float() if bias else None, clamp=clamp)
    layer.name = "q"
    xs = [torch.randn(T, K, generator=g, device="cuda").bfloat16() for T in (3, 100)]
    want = [layer(x) for x in xs]
    say("copy", K, bias, clamp)
    other = how(layer)
    mine = other._weights
    assert mine[:1] + mine[2:3] == (other.codes.data_ptr(), other.scale.data_ptr()) and mine[3] == (other.bias.data_ptr() if bias else 0)
    assert (other.N, other.K, other.device, other.clamp, other.name) == (70, K, layer.device, clamp, "q")
    if how is not copy.copy:  # a plain copy shares its tensors
        layer.codes.zero_()
        layer.scale.zero_()
    del layer
    assert all(torch.equal(other(x), y) for x, y in zip(xs, want))
