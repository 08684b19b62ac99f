"""Python binding of the operators around the compressed linear layers
(include/cl_serving.h): rotary positions, the quantised K/V cache, attention of
drafted tokens over it, and log probabilities of given tokens.

Argument checks and marshalling only; every step runs in the HIP library, on
torch's current stream of the tensors' device.  Index tensors are int32.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

SERVING_SYMBOLS = ["cl_rope_table", "cl_rope", "cl_kv_append", "cl_kv_read", "cl_tree_attention_work_bytes",
                   "cl_tree_attention", "cl_recording", "cl_token_logprobs", "cl_call"]


class UnknownName(ValueError, KeyError):
    """An argument that names none of the choices."""

    __str__ = ValueError.__str__


class _Names(dict):
    def __missing__(self, name):
        raise UnknownName(f"{name!r} is none of {list(self)}")


ROPE_LAYOUT = _Names(half=0, interleaved=1)
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
KV_KIND = {"int8": 0, "int4": 1}
COUNTER_BYTES = 262144  # CL_ATTENTION_COUNTER_BYTES
_ROOM = 32 << 20        # bytes that a workspace may have beyond what its call needs
_ENDED = 4              # recordings that a cache may list before it asks which have ended


class cl_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def declare(L):
    """Argument types of the entry points, on the loaded library."""
    p, i, q, d = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    cache = ctypes.POINTER(cl_kv_cache)
    L.cl_rope_table.argtypes = [i, i, d, i, d, i, d, d, p, p]
    L.cl_rope.argtypes = [p, i, q, q, i, i, i, p, p, i, i, i, p, i, q, q, p]
    L.cl_kv_append.argtypes = [cache, p, p, i, i, q, q, q, q, p, p, p, i, i, i, p]
    L.cl_kv_read.argtypes = [cache, p, i, p, p, i, p]
    L.cl_tree_attention_work_bytes.argtypes = [i] * 6
    L.cl_tree_attention.argtypes = [p, i, q, q, i, i, cache, p, i, i, p, p, i, i, p, i, ctypes.c_float, p, p,
                                    ctypes.c_size_t, p]
    L.cl_recording.argtypes = [p, ctypes.POINTER(ctypes.c_uint64)]
    L.cl_token_logprobs.argtypes = [p, i, q, i, i, p, i, p, p, i, p, p, p]
    L.cl_call.argtypes = [i, ctypes.c_char_p]
    for name in SERVING_SYMBOLS:
        getattr(L, name).restype = ctypes.c_size_t if name.endswith("_bytes") else ctypes.c_int


# cl_call's entries and how their arguments are packed: 0.3 us a call, where ctypes takes 0.8 for 17 of them
_ROPE, _APPEND, _READ, _ATTENTION, _LOGPROBS = range(5)
_pack_rope, _pack_append, _pack_read, _pack_attention, _pack_logprobs = (
    struct.Struct(f).pack for f in ("17q", "16q", "7q", "16qd4q", "13q"))

_torch = None
_lib = None
_empty = _current_device = _raw_stream = _capturing = _i32 = None
_DT: dict = {}


def _setup():
    """torch and the library, loaded at the first call (importing the package needs neither)."""
    global _torch, _lib, _empty, _current_device, _raw_stream, _capturing, _i32
    if _lib is None:
        import torch

        from . import lib
        _torch, _empty, _i32 = torch, torch.empty, torch.int32
        # the device's number without a check that torch is set up (0.2 us of a call: the tensors are there), the stream's
        # address without a Stream object around it (1.8 us), where torch has those
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)
        _capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
        _DT.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
        _lib = lib()
    return _lib


def _check(st: int, where: str):
    if st != 0:
        from . import _check as check
        check(st, where)


def _stream(dev):
    """torch's current stream on `dev`; the library launches on the current device, so that has to be it."""
    index = dev.index
    if index != _current_device():
        raise ValueError(f"tensors on {dev}, but the current device is cuda:{_current_device()}")
    return _raw_stream(index)


def _index(t, n, dev, what):
    """The address of an int32 tensor of n elements on `dev`."""
    if t.dtype is not _i32 or t.numel() != n or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of {n} elements on {dev}")
    return t.data_ptr()


def _heads3(x, what):
    """A [tokens, heads, dim] tensor of 16 or 32 bits with contiguous channels (copied if they are not)."""
    if x.dim() != 3 or x.dtype not in _DT or not x.is_cuda:
        raise ValueError(f"{what} must be a float16, bfloat16 or float32 [tokens, heads, dim] tensor on a ROCm device")
    return x if x.stride(2) == 1 else x.contiguous()


def _table(table, dev):
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2 or table.dtype is not _torch.float32 or table.device != dev \
            or not table.is_contiguous():
        raise ValueError(f"table must be a contiguous float32 [positions, rot / 2, 2] tensor on {dev} (see rope_table)")
    return table.data_ptr(), shape[0], 2 * shape[1]


def rope_table(positions: int, rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               trained: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Cosines and sines of `positions` positions for a rotation over `rot` channels (cl_rope_table): a
    float32 tensor [positions, rot / 2, 2].  scaling 'none', 'linear', 'ntk' or 'yarn' (by `factor`;
    'yarn' also reads `trained`, `beta_fast` and `beta_slow`)."""
    L = _setup()
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALING)}")
    dev = _torch.device("cuda", _torch.cuda.current_device()) if device is None else _torch.device(device)
    if positions < 1 or rot < 2 or rot % 2:
        raise ValueError("positions >= 1 and an even rot >= 2 are wanted")
    out = _torch.empty((positions, rot // 2, 2), dtype=_torch.float32, device=dev)
    _check(L.cl_rope_table(positions, rot, base, ROPE_SCALING[scaling], factor, trained, beta_fast, beta_slow,
                           out.data_ptr(), _stream(out.device)), "cl_rope_table")
    return out


def rope(x, positions, table, layout: str = "half", out=None, out_dtype=None):
    """Rotary positions (cl_rope): x [tokens, heads, dim] float16, bfloat16 or float32 (any token and head
    strides, so a view of a qkv output will do), positions int32 [tokens], table from `rope_table`; the
    first 2 * table.shape[1] channels are rotated, the others copied.  Returns `out`, or a new
    contiguous tensor of `out_dtype` (x's type by default).  `out` may be x."""
    L = _lib or _setup()
    x = _heads3(x, "x")
    dev, shape = x.device, x.shape
    T, H, D = shape
    xt, xh, _ = x.stride()
    if out is None:
        out = _empty(T, H, D, dtype=out_dtype or x.dtype, device=dev)  # sizes as numbers: 0.8 us less than as a shape
        yt, yh = H * D, D
    else:
        yt, yh, one = out.stride() if out.dim() == 3 else (0, 0, 0)
        if out.shape != shape or out.device != dev or one != 1 or (out_dtype or out.dtype) != out.dtype:
            raise ValueError(f"out must be a {tuple(shape)} tensor on {dev} with contiguous channels")
    if out.dtype not in _DT:
        raise ValueError("the output must be float16, bfloat16 or float32")
    tp, rows, rot = _table(table, dev)
    st = L.cl_call(_ROPE, _pack_rope(
        x.data_ptr(), _DT[x.dtype], xt, xh, T, H, D, _index(positions, T, dev, "positions"), tp, rows, rot,
        ROPE_LAYOUT[layout], out.data_ptr(), _DT[out.dtype], yt, yh, _stream(dev)))
    if st:
        _check(st, "cl_rope")
    return out


class KVCache:
    """A paged, quantised K/V cache on one GPU (cl_kv_cache): kind 'int8' (a scale to each token and head)
    or 'int4' (a scale to each 32 channels).  Slot s is place s % page_size of page s // page_size.

    Either sizes are given and the cache allocates its tensors, or the four tensors are:
    k, v uint8 [pages, heads, page_size, dim or dim / 2]; k_scale, v_scale float16 [pages, heads,
    page_size] or [pages, heads, page_size, dim / 32].  It also keeps a workspace of `tree_attention` for
    each stream it is called on, and one for each recording (torch.cuda.graph) that it is called in: a replay may
    run on any stream, next to other calls.  A recording's lies in its graph's own memory, and goes with it.
    """

    def __init__(self, pages: int = 0, page_size: int = 64, heads: int = 1, dim: int = 128, kind: str = "int8",
                 device=None, k=None, v=None, k_scale=None, v_scale=None):
        _setup()
        torch = _torch
        if kind not in KV_KIND:
            raise ValueError(f"kind must be one of {list(KV_KIND)}")
        four = (k, v, k_scale, v_scale)
        if all(t is None for t in four):
            dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
            width = dim if kind == "int8" else dim // 2
            tail = () if kind == "int8" else (dim // 32,)
            k, v = (torch.zeros((pages, heads, page_size, width), dtype=torch.uint8, device=dev) for _ in range(2))
            k_scale, v_scale = (torch.zeros((pages, heads, page_size) + tail, dtype=torch.float16, device=dev)
                                for _ in range(2))
        elif any(t is None for t in four):
            raise ValueError("k, v, k_scale and v_scale are given together")
        if k.dim() != 4:
            raise ValueError("k must be uint8 [pages, heads, page_size, dim or dim / 2]")
        pages, heads, page_size, width = k.shape
        dim = width if kind == "int8" else 2 * width
        tail = () if kind == "int8" else (dim // 32,)
        for t, shape, dt in ((k, k.shape, torch.uint8), (v, k.shape, torch.uint8),
                             (k_scale, (pages, heads, page_size) + tail, torch.float16),
                             (v_scale, (pages, heads, page_size) + tail, torch.float16)):
            if tuple(t.shape) != tuple(shape) or t.dtype != dt or t.device != k.device or not t.is_cuda \
                    or not t.is_contiguous():
                raise ValueError(f"a cache tensor must be a contiguous {dt} tensor {tuple(shape)} on one ROCm device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kind, self.pages, self.page_size, self.heads, self.dim = kind, pages, page_size, heads, dim
        self.device = k.device
        self._desc = cl_kv_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, page_size,
                                 heads, dim, KV_KIND[kind], 0)
        self._ref = ctypes.addressof(self._desc)
        self._work: dict = {}   # by stream, or stream and recording: address and bytes of the workspace
        self._keep: dict = {}   # their tensors
        self._recorded = 0      # how many of them are recordings'

    def append(self, k, v, slots, positions=None, table=None, layout: str = "half"):
        """Quantise new keys and values [tokens, heads, dim] into `slots` (int32 [tokens]; a slot outside the
        cache, -1 say, stores nothing).  With `table` (and int32 `positions`) the keys are rotated on
        the way, from unrounded results, as `rope` would."""
        k, v, dev = _heads3(k, "k"), _heads3(v, "v"), self.device
        shape, dt = k.shape, k.dtype
        if v.shape != shape or v.dtype is not dt or k.device != dev or v.device != dev \
                or shape[1] != self.heads or shape[2] != self.dim:
            raise ValueError(f"k and v must be [tokens, {self.heads}, {self.dim}] of one type on {dev}")
        T = shape[0]
        pp = tp = rows = rot = 0
        if table is not None:
            tp, rows, rot = _table(table, dev)
            if positions is None:
                raise ValueError("a table needs positions")
            pp = _index(positions, T, dev, "positions")
        kt, kh, _ = k.stride()
        vt, vh, _ = v.stride()
        st = _lib.cl_call(_APPEND, _pack_append(
            self._ref, k.data_ptr(), v.data_ptr(), _DT[dt], T, kt, kh, vt, vh, _index(slots, T, dev, "slots"), pp, tp,
            rows, rot, ROPE_LAYOUT[layout], _stream(dev)))
        if st:
            _check(st, "cl_kv_append")

    def read(self, slots, dtype=None):
        """The stored keys and values of `slots` (int32 [n]): two tensors [n, heads, dim] of `dtype` (float16
        by default), zeros for a slot outside the cache."""
        dev = self.device
        dtype = dtype or _torch.float16
        if dtype not in _DT:
            raise ValueError("dtype must be float16, bfloat16 or float32")
        n = slots.numel()
        k, v = _empty(2, n, self.heads, self.dim, dtype=dtype, device=dev).unbind(0)
        st = _lib.cl_call(_READ, _pack_read(self._ref, _index(slots, n, dev, "slots"), n, k.data_ptr(), v.data_ptr(),
                                            _DT[dtype], _stream(dev)))
        if st:
            _check(st, "cl_kv_read")
        return k, v

    def _recording(self, stream):
        """Whose workspace a call that is recorded on `stream` takes.  It is the recording's even where the stream has
        one, with which nothing orders the replays; what clears it runs with them."""
        recording = ctypes.c_uint64()
        _check(_lib.cl_recording(stream, ctypes.byref(recording)), "cl_recording")
        return stream, recording.value

    def _let_go(self):
        """Drops the workspaces of recordings that have ended.  torch allocated them from their graph's memory, which
        stays the graph's until it is deleted."""
        now = ctypes.c_uint64()
        for key in [k for k in self._work if type(k) is tuple]:
            if _lib.cl_recording(key[0], ctypes.byref(now)) or now.value != key[1]:
                if self._work.pop(key, None):  # another thread may have been here
                    self._keep.pop(key, None)
                    self._recorded -= 1

    def _workspace(self, sizes, key):
        """Address and bytes of a workspace for these sizes, of a stream or of a recording on it.  An outgrown one can
        go at once: its memory is given out again on its stream only, after the calls that use it."""
        if self._recorded >= _ENDED and key not in self._work:
            self._let_go()
        need = _lib.cl_tree_attention_work_bytes(*sizes)
        size = need + min(need, _ROOM)
        work = self._keep[key] = _empty(size, dtype=_torch.uint8, device=self.device)
        work[:COUNTER_BYTES].zero_()  # the calls leave them so
        if type(key) is tuple and key not in self._work:
            self._recorded += 1
        self._work[key] = work.data_ptr(), size
        return self._work[key]


def tree_attention(q, cache: KVCache, block_table, ctx_lens, cu_q, max_q: int, max_ctx: Optional[int] = None,
                   tree_mask=None, scale: Optional[float] = None, out=None):
    """Attention of each sequence's newest tokens over its cached keys and values (cl_tree_attention).

    q [tokens, q_heads, dim] float16 or bfloat16: the new tokens of all sequences, those of sequence b in
    rows cu_q[b] .. cu_q[b + 1] (int32 [sequences + 1]); they are already in the cache, after its
    ctx_lens[b] (int32 [sequences]) older tokens.  block_table int32 [sequences, width] names the
    cache pages.  tree_mask int64 [tokens, words]: bit i of a row is set where the row's token sees
    new token i of its sequence (None: the tokens form a chain).  max_q is at least every sequence's number
    of new tokens (at most 256); max_ctx the longest context, which sizes the launch (default: what the
    block table holds).  Returns [tokens, q_heads, dim] of q's type: `out`, or a new tensor.  Rows of a sequence
    with more than max_q new tokens, and rows past the last sequence, are not written: in a new tensor they hold
    whatever was in memory."""
    L = _lib or _setup()
    dev = cache.device
    shape, dt = q.shape, _DT.get(q.dtype, 2)
    if len(shape) != 3 or q.device != dev or shape[2] != cache.dim or dt == 2:
        raise ValueError(f"q must be a float16 or bfloat16 [tokens, q_heads, {cache.dim}] tensor on {dev}")
    qt, qh, one = q.stride()
    qp = q.data_ptr()
    if one != 1 or qt % 8 or qh % 8 or qp % 16:
        q = q.clone(memory_format=_torch.contiguous_format)  # contiguous() leaves one that only lies at an odd address
        qt, qh, _ = q.stride()
        qp = q.data_ptr()
    T, H, D = shape
    B = ctx_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be int32 [{B}, width]")
    width = block_table.shape[1]
    words = mp = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2 or tree_mask.dtype is not _torch.int64 or tree_mask.device != dev \
                or tree_mask.shape[0] != T or not tree_mask.is_contiguous():
            raise ValueError(f"tree_mask must be a contiguous int64 [{T}, words] tensor on {dev}")
        words, mp = tree_mask.shape[1], tree_mask.data_ptr()
    if out is None:
        out = _empty(T, H, D, dtype=q.dtype, device=dev)
    elif out.shape != shape or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape and type")
    if max_ctx is None:
        max_ctx = width * cache.page_size
    args = (qp, dt, qt, qh, T, H, cache._ref, _index(block_table, B * width, dev, "block_table"), width, B,
            _index(ctx_lens, B, dev, "ctx_lens"), _index(cu_q, B + 1, dev, "cu_q"), max_q, max_ctx, mp, words,
            1.0 / D ** 0.5 if scale is None else scale, out.data_ptr())
    stream = _stream(dev)
    if _capturing():
        key = cache._recording(stream)
    else:
        key = stream
        if cache._recorded:
            cache._let_go()
    st = L.cl_call(_ATTENTION, _pack_attention(*args, *cache._work.get(key, (0, 0)), stream))
    if st == -3:  # the workspace is too small for these sizes: make a larger one, once
        work = cache._workspace((B, H, cache.heads, D, max_q, max_ctx), key)
        st = L.cl_call(_ATTENTION, _pack_attention(*args, *work, stream))
    if st:
        _check(st, "cl_tree_attention")
    return out


def token_logprobs(logits, ids, top_k: int = 0):
    """Log probabilities of given tokens (cl_token_logprobs): logits [rows, vocab] float16, bfloat16 or float32,
    ids int32 [rows, given].  Returns (logp float32 [rows, given], entropy float32 [rows]) and, with top_k > 0
    (at most 32), top_ids int32 [rows, top_k] and top_logp float32 [rows, top_k]: the largest logits first,
    equal ones by the lower id.  An id outside the vocabulary gives NaN.  The outputs are parts of one allocation,
    which lives as long as any of them."""
    L = _lib or _setup()
    shape, dt = logits.shape, _DT.get(logits.dtype)
    if len(shape) != 2 or dt is None or not logits.is_cuda:
        raise ValueError("logits must be a float16, bfloat16 or float32 [rows, vocab] tensor on a ROCm device")
    row, one = logits.stride()
    if one != 1:
        logits = logits.contiguous()
        row = logits.stride(0)
    dev = logits.device
    T, V = shape
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be int32 [{T}, given]")
    C = ids.shape[1]
    ip = _index(ids, T * C, dev, "ids")
    # the outputs are pieces of one allocation
    n = T * C
    buf = _empty(n + T + 2 * T * max(top_k, 0), dtype=_torch.float32, device=dev)
    at = buf.data_ptr()
    logp, entropy = buf.as_strided((T, C), (C, 1), 0), buf.as_strided((T,), (1,), n)
    top_ids = top_logp = None
    tip = tlp = 0
    if top_k > 0:
        top_logp = buf.as_strided((T, top_k), (top_k, 1), n + T)
        top_ids = buf.view(_i32).as_strided((T, top_k), (top_k, 1), n + T + T * top_k)
        tlp = at + 4 * (n + T)
        tip = tlp + 4 * T * top_k
    st = L.cl_call(_LOGPROBS, _pack_logprobs(logits.data_ptr(), dt, row, T, V, ip, C, at, at + 4 * n, top_k, tip, tlp,
                                             _stream(dev)))
    if st:
        _check(st, "cl_token_logprobs")
    return (logp, entropy, top_ids, top_logp) if top_k else (logp, entropy)
