"""The 8-bit integer layer's outputs to the last bit (numpy, no library code): its sums are exact, and each rounding after them is stated."""
import numpy as np


def sums(q, w):
    """Exact sums of products (below 2^31, so that 64-bit floats hold them), as float64."""
    return np.rint(q.astype(np.float64) @ w.astype(np.float64).T)


def outputs(acc, s, ws, bias=None):
    """float32 outputs: the sum rounded, then each product with a scale, then the sum with the bias."""
    v = acc.astype(np.float32) * np.asarray(s, np.float32)[:, None]
    v = v * np.asarray(ws, np.float32)
    return v if bias is None else v + np.asarray(bias, np.float32)


def fused(acc, s, ws, bias):
    """What a fused multiply-add in the place of the last product and sum would give (64 bits hold the product)."""
    v = (acc.astype(np.float32) * np.asarray(s, np.float32)[:, None]).astype(np.float64)
    return (v * np.asarray(ws, np.float64) + np.asarray(bias, np.float64)).astype(np.float32)


def weights(r, N, K):
    """Codes, scales and biases that are as large as the products, so that a sum that is rounded once less is seen."""
    w = r.integers(-127, 128, (N, K)).astype(np.int8)
    size = 1 / (127.0 * 127 * K ** 0.5)
    return w, (r.uniform(0.5, 2, N) * size).astype(np.float32), r.normal(0, 1, N).astype(np.float32)


def activations(r, T, K):
    return r.integers(-127, 128, (T, K)).astype(np.int8), r.uniform(1, 50, T).astype(np.float32)
