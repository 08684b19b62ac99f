"""Plain 64-bit references and inputs for the serving operators' tests (numpy, no library code)."""
import numpy as np

U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # unit roundoffs


def torch_dtype(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def to_bf16(a):
    """float32 values rounded to bf16 (nearest-even), as float32."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


# ------------------------------------------------------------------- rotary
def rope_table(P, rot, base=10000.0, scaling="none", factor=1.0, trained=4096, fast=32.0, slow=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    m = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    w = base ** (-2.0 * i / rot)
    if scaling == "linear":
        w = w / factor
    if scaling == "yarn":
        at = [rot * np.log(trained / (b * 2 * np.pi)) / (2 * np.log(base)) for b in (fast, slow)]
        lo, hi = np.clip(np.floor(at[0]), 0, rot - 1), np.clip(np.ceil(at[1]), 0, rot - 1)
        g = 1.0 - np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        w = w / factor * (1 - g) + w * g
        m = 0.1 * np.log(factor) + 1.0
    a = np.arange(P, dtype=np.float64)[:, None] * w
    return np.stack([np.cos(a) * m, np.sin(a) * m], -1)


def rotate(x, pos, table, layout):
    """x [T, H, D] rotated in x's own precision (float32: every product and sum rounded; float64: the formula)."""
    y = x.copy()
    n = table.shape[1]
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    c, s = (table[pos][:, None, :, j].astype(x.dtype) for j in (0, 1))
    u, v = x[..., a], x[..., b]
    y[..., a] = u * c - v * s
    y[..., b] = v * c + u * s
    return y


# -------------------------------------------------------------------- cache
def quantise(v, kind):
    """(codes int [..., D], scales float16) of float32 values, by the format's rule in fp32."""
    v = np.asarray(v, np.float32)
    v = np.where(np.isnan(v), np.float32(0), v)
    most, width, big = (127, v.shape[-1], 65504.0) if kind == "int8" else (7, 32, 8192.0)
    g = v.reshape(*v.shape[:-1], -1, width)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore", under="ignore"):
        s = np.minimum(np.abs(g).max(-1, keepdims=True) / np.float32(most), np.float32(big))
        if kind == "int4":
            s = to_bf16(s)
        s = s.astype(np.float16)
        f = s.astype(np.float32)
        r = np.where(f > 0, np.float32(1) / f, np.float32(0))
        q = np.where(f > 0, np.clip(np.rint(g * r), -most, most), 0)
    q = q.astype(np.int32).reshape(v.shape)
    s = s[..., 0]
    return q, (s[..., 0] if kind == "int8" else s)


def codes_to_bytes(q, kind):
    if kind == "int8":
        return (q + 128).astype(np.uint8)
    n = (q + 8).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def stored(q, s, kind):
    """float64 values of codes and scales."""
    s = s.astype(np.float64)
    return q * (s[..., None] if kind == "int8" else np.repeat(s, 32, -1))


# ---------------------------------------------------------------- attention
def attention(q, k, v, see, scale):
    """q [t, D], k and v [n, D] float64, see [t, n] -> (o, sum_j p_j |v_j|, largest sum_i |q_i k_i| scale) per row.
    The second has one term more, for probabilities below fp16's normal range, which are kept to 2^-35 of the largest:
    2^-24 of the largest times sum_j |v_j|, as attention_tolerance weighs it with 2^-11."""
    s = (q @ k.T) * scale
    s = np.where(see, s, -np.inf)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = p.sum(-1, keepdims=True)
    p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    mag = np.abs(q) @ np.abs(k).T * abs(scale)
    lost = 2.0 ** -24 * p.max(-1, keepdims=True, initial=0.0) * (see @ np.abs(v).max(-1, keepdims=True))
    return p @ v, p @ np.abs(v) + lost, np.where(see, mag, 0).max(-1, keepdims=True, initial=0.0)


def attention_tolerance(o, absv, mag, n, D, dtype):
    """Bound of |kernel - o|.  The output is rounded once (unit roundoff u of its type, and below fp16's normal
    range half its smallest step, 2^-25).  A score's fp32
    sum of D products, its scale factors and exp2's argument put (D + 8) 2^-24 of sum |q k| into the
    exponent, which moves each probability by that and, through the denominator, once more; each probability
    is rounded to fp16 (2^-11), and the fp32 sums over n keys, exp2 and the join add (n + 64) 2^-24."""
    rel = 2.0 ** -11 + 2.0 * (D + 8) * 2.0 ** -24 * mag + 2 * (n + 64) * 2.0 ** -24
    return U[dtype] * np.abs(o) + 1.05 * rel * absv + 1e-7 * absv + (2.0 ** -25 if dtype == "f16" else 1e-30)


# ----------------------------------------------------------------- logprobs
def logprobs(x, ids, k):
    """float64 (logp, entropy, top_ids, top_logp, W) of x [T, V]; W = sum_j |x_j - m| p_j."""
    x = x.astype(np.float64)
    T, V = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        m = np.where(np.isnan(x).any(-1, keepdims=True), np.nan, x.max(-1, keepdims=True))
        d = x - m
        e = np.exp(d)
        l = e.sum(-1, keepdims=True)
        w = np.where(np.isneginf(d), 0.0, d * e).sum(-1, keepdims=True)
        lse = np.log(l)
        ent = (lse - w / l)[:, 0]
        ok = (ids >= 0) & (ids < V)
        logp = np.where(ok, np.take_along_axis(d, np.where(ok, ids, 0), 1) - lse, np.nan)
        key = np.where(np.isnan(x), np.inf, x)
        nan = np.isnan(x)
        top = np.stack([np.lexsort((np.arange(V), -key[t], ~nan[t]))[:k] for t in range(T)]) if T else \
            np.zeros((0, k), np.int64)
        return logp, ent, top, np.take_along_axis(d, top, 1) - lse, (np.abs(w) / l)[:, 0]


def logprob_tolerance(x, logp):
    """Bound of the fp32 log probabilities: x - m, log l and their difference round at their own magnitudes; l is
    a sum of V terms (at most V / 64 + 64 roundings deep), each off by its exponent's rounding."""
    f = x[np.isfinite(x)]
    big = np.abs(f).max(initial=0.0)
    return 2.0 ** -24 * (8 * big + 8 * np.abs(logp) + x.shape[1] / 64 + 64)
