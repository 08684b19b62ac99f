"""Plain references for the 8-bit integer layer's tests (numpy, no library code)."""
import numpy as np

from serving_ref import U

LEAST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half of a type's smallest step


def quantise(x, clamp=0.0):
    """(codes int64 [T, K], scale float32 [T]) of float32 values, by the rule in fp32."""
    x = np.asarray(x, np.float32)
    if clamp:
        x = np.where(np.abs(x) > clamp, np.copysign(np.float32(clamp), x), x)
    a = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    any_ = ~bad & (a >= np.float32(2.0 ** -100))
    with np.errstate(all="ignore"):
        s = np.where(any_, a * np.float32(1.0 / 127.0), np.float32(0)).astype(np.float32)
        r = np.where(any_, np.float32(1) / s, np.float32(0)).astype(np.float32)
        q = np.clip(np.rint(x * r[:, None]), -127, 127)
    q = np.where(any_[:, None], q, 0).astype(np.int64)
    return q, np.where(bad, np.float32(np.nan), s).astype(np.float32)


def product(q, s, w, ws, bias=None):
    """float64 y and a bound's magnitudes |sum| s ws."""
    acc = (q.astype(np.int64) @ w.astype(np.int64).T).astype(np.float64) if q.shape[1] < 64 else \
        np.rint(q.astype(np.float64) @ w.astype(np.float64).T)  # sums below 2^31: exact in 64-bit floats
    p = acc * s.astype(np.float64)[:, None] * ws.astype(np.float64)
    return (p if bias is None else p + bias.astype(np.float64)), np.abs(p)


def tolerance(y, p, bias, dtype):
    """The sum rounded to fp32, two products, the sum with the bias (2^-24 each), then y's type."""
    b = 0.0 if bias is None else np.abs(bias.astype(np.float64))
    u = 2.0 ** -24
    t = 3.001 * u * p + (1.001 * u * (p + b) if bias is not None else 0.0) + 4 * LEAST["f32"]
    return t + (U[dtype] * 1.001 * (np.abs(y) + t) + LEAST[dtype] if dtype != "f32" else 0.0)
