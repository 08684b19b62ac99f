"""The inputs that the 8-bit integer layer's bits are compared on tell a fused sum from a rounded one (no GPU)."""
import numpy as np
import pytest

import int8_bits as ref


@pytest.mark.parametrize("T,K,N", [(1, 77, 300), (5, 300, 77), (300, 129, 500)])
def test_a_fused_sum_would_be_seen(T, K, N):
    r = np.random.default_rng(K)
    w, ws, bias = ref.weights(r, N, K)
    q, s = ref.activations(r, T, K)
    acc = ref.sums(q, w)
    assert np.array_equal(acc.astype(np.int64), q.astype(np.int64) @ w.astype(np.int64).T)
    differ = ref.outputs(acc, s, ws, bias) != ref.fused(acc, s, ws, bias)
    assert differ.mean() > 0.05
