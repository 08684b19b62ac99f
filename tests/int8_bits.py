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


# Sizes by how a product is cut, each with steps enough (in each part of K) for a ring of buffers to go round twice, K odd and the last
# tiles ragged: (tokens, K, N): tile, whether K is in parts, which tiles are cut in halves of 128 tokens.
PLANS = {
    (408, 729, 22183): ("256x256", False, "none"),
    (261, 781, 13157): ("256x256", False, "all"),
    (1354, 891, 24653): ("256x256", False, "some"),  # 512 whole ones, then 70 in halves, of which some have no tokens
    (2319, 883, 15207): ("256x256", False, "some"),  # in two runs of token tiles
    (193, 2925, 17119): ("256x256", True, "none"),
    (261, 725, 22125): ("256x192", False, "none"),
    (129, 6529, 5943): ("256x192", True, "none"),
    (259, 779, 18405): ("256x128", False, "none"),
    (67, 9481, 11087): ("256x128", True, "none"),
    (69, 1031, 17121): ("128x128", False, "none"),
    (72, 18413, 1187): ("128x128", True, "none"),
    (67, 789, 8327): ("128x64", False, "none"),
    (17, 6197, 5497): ("128x64", True, "none"),
    (66, 1089, 5603): ("64x64", False, "none"),
    (165, 18419, 139): ("64x64", True, "none"),
    (65, 1077, 137): ("64x32", False, "none"),
    (67, 18427, 131): ("64x32", True, "none"),
}
BUFFERS = {"256x256": 2, "256x192": 2, "256x128": 3, "128x128": 4, "128x64": 3, "64x64": 4, "64x32": 4}  # halves have one more

# Layers whose rows are computed by many tiles, and the numbers of tokens.
ROWS = {(3001, 9001): (1, 16, 40, 65, 200, 500, 777, 1300), (1411, 2050): (1, 16, 40, 100, 300, 777, 1300, 2049),
        (5001, 4100): (7, 40, 65, 300, 500, 1300)}
