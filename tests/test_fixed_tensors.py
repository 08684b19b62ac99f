"""Layers and pools hold their tensors' addresses from their construction, so that putting others in their place is refused (no GPU)."""
import pytest
import torch

import compressed_linear_amd as cla


def made(cls, **attributes):
    """An object as its constructor leaves it, but for tensors on a GPU."""
    it = object.__new__(cls)
    it.__dict__.update(attributes)
    return it


def test_a_layer_refuses_other_weights():
    codes, scale, bias = object(), object(), object()
    layer = made(cla.Int8Linear, codes=codes, scale=scale, bias=bias, clamp=None, N=4, K=128, device="cuda:0")
    for name, other in (("codes", object()), ("scale", object()), ("bias", None), ("clamp", 1.0), ("N", 3), ("K", 64), ("device", "cuda:1")):
        old = getattr(layer, name)
        with pytest.raises(AttributeError, match=name):
            setattr(layer, name, other)
        assert getattr(layer, name) is old
        setattr(layer, name, old)  # what `layer.bias += 1` does once the sum is in place
    layer.name = "q"  # a program's own
    assert layer.name == "q"



def test_a_pool_refuses_other_tensors():
    pool = made(cla.PagePool, block_table=object(), lens=[1, 2], refs=object(), left_out=object(), device="cuda:0", sequences=3, width=4,
                pages=8, page_size=16)
    for name in list(pool.__dict__):
        old = getattr(pool, name)
        with pytest.raises(AttributeError, match=name):
            setattr(pool, name, object())
        assert getattr(pool, name) is old
    lens = pool.lens
    pool.lens += [3]  # in place
    assert pool.lens is lens and lens == [1, 2, 3]


def test_a_copy_of_a_layer_is_made_from_its_weights():
    """A deep copy and a pickled layer have tensors of their own, so that the addresses of the first one's must not come along."""
    codes, scale, bias = torch.zeros(4, 128, dtype=torch.int8), torch.ones(4), torch.ones(4)
    layer = made(cla.Int8Linear, codes=codes, scale=scale, bias=bias, clamp=2.0, N=4, K=100, device="cuda:0",
                 _weights=(codes.data_ptr(), 128, scale.data_ptr(), bias.data_ptr(), 4, 100))
    how, what, *rest = layer.__reduce_ex__(4)
    assert how is cla.Int8Linear and not any(rest)
    assert torch.equal(what[0], codes[:, :100]) and what[1] is scale and what[2] is bias and what[3] == 2.0
