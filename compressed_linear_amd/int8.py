"""Python binding of the linear layer in 8-bit integers (include/cl_int8.h): weights with a scale to each
output channel, activations quantised on the way in with a scale to each token.

Argument checks and marshalling only; every step runs in the HIP library, on torch's current stream of the
tensors' device.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

from . import serving as _s

INT8_SYMBOLS = ["cl_int8_quant", "cl_int8_linear", "cl_int8_work_bytes", "cl_int8_forward"]
MOST_K = 131071

_QUANT, _LINEAR, _FORWARD = 24, 25, 26
_pack_quant, _pack_linear, _pack_forward = (struct.Struct(f).pack for f in ("5qd4q", "16q", "4qd12q"))


def declare(L):
    """Argument types of the entry points, on the loaded library."""
    p, i, q, f, z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    L.cl_int8_quant.argtypes = [p, i, q, i, i, f, p, q, p, p]
    L.cl_int8_linear.argtypes = [p, q, p, i, p, q, p, p, i, i, p, i, q, p, z, p]
    L.cl_int8_work_bytes.argtypes = [i, i, i, i]
    L.cl_int8_forward.argtypes = [p, i, q, i, f, p, q, p, p, i, i, p, i, q, p, z, p]
    for name in INT8_SYMBOLS:
        getattr(L, name).restype = z if name.endswith("_bytes") else ctypes.c_int


def _padded(K):
    return -(-K // 128) * 128


def _rows2(x, K, dev, what):
    """A [rows, K] tensor of 16 or 32 bits with contiguous columns (copied if they are not), and its row stride."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dim() != 2 or x.dtype not in _s._DT or not x.is_cuda or (K is not None and x.shape[1] != K) \
            or (dev is not None and x.device != dev):
        raise ValueError(f"{what} must be a float16, bfloat16 or float32 [rows, {K or 'K'}] tensor on "
                         f"{dev or 'a ROCm device'}")
    row, one = x.stride()
    if one != 1 and x.shape[1] != 1:
        x = x.contiguous()
        row = x.stride(0)
    return x, row


def _clamp(clamp):
    c = 0.0 if clamp is None else float(clamp)
    if clamp is not None and not 0.0 < c < 3.4e38:
        raise ValueError("clamp must be positive and finite (None: no clamp)")
    # The entries take 0 as no clamp, which a clamp below the least float would become; all clamps below 2^-100 give zeros.
    return max(c, 2.0 ** -126) if clamp is not None else 0.0


def quantize_rows(x, clamp: Optional[float] = None):
    """Rows of values to 8-bit codes with a scale to each row (cl_int8_quant): x [rows, K] float16, bfloat16 or float32,
    any row stride.  Returns (codes int8 [rows, K], scale float32 [rows]); codes are the first K columns of
    rows of a multiple of 128 bytes.  Activations by token (clamp: clipped to [-clamp, clamp] before), or weights by
    output channel."""
    L = _s._lib or _s._setup()
    x, row = _rows2(x, None, None, "x")
    T, K = x.shape
    if not 1 <= K <= MOST_K:
        raise ValueError(f"rows of 1 to {MOST_K} values are wanted")
    dev, width = x.device, _padded(K)
    codes = _s._empty(T, width, dtype=_s._torch.int8, device=dev)
    scale = _s._empty(T, dtype=_s._torch.float32, device=dev)
    st = L.cl_call(_QUANT, _pack_quant(x.data_ptr(), _s._DT[x.dtype], row, T, K, _clamp(clamp), codes.data_ptr(), width,
                                       scale.data_ptr(), _s._stream(dev)))
    if st:
        _s._check(st, "cl_int8_quant")
    return codes[:, :K], scale


def _whole_rows(codes):
    """Whether a [rows, K] int8 tensor's rows are readable up to the next multiple of 128 bytes, as the kernels read them."""
    T, K = codes.shape
    row, one = codes.stride()
    if T == 1:
        row = max(row, _padded(K)) // 128 * 128
    end = codes.storage_offset() + (T - 1) * row + _padded(K)
    return (one == 1 or K == 1) and row % 128 == 0 and K <= row <= 1 << 23 and codes.data_ptr() % 16 == 0 \
        and end <= codes.untyped_storage().nbytes(), row


class Int8Linear(_s._Fixed):
    """A linear layer in 8-bit integers on one GPU: y[t, n] = (sum_k a[t, k] w[n, k]) s[t] scale[n] + bias[n], the
    sum exact in 32-bit integers, a and s the token's codes and scale (quantize_rows).

    codes int8 [N, K] and scale float32 [N] are the weights, by output channel; bias float32 [N]; clamp: the
    activations are clipped to [-clamp, clamp] before they are quantised.  Codes whose K is a multiple of 128 are used as they
    are; others are copied into rows padded with zeros.  What a layer was made with stays (its tensors' values may change); a
    copy, deep or pickled, is a layer of its own.
    """

    _fixed = frozenset(("codes", "scale", "bias", "clamp", "N", "K", "device"))

    def __init__(self, codes, scale, bias=None, clamp: Optional[float] = None):
        _s._setup()
        torch = _s._torch
        if codes.dim() != 2 or codes.dtype is not torch.int8 or not codes.is_cuda:
            raise ValueError("codes must be an int8 [N, K] tensor on a ROCm device")
        N, K = codes.shape
        if N < 1 or not 1 <= K <= MOST_K:
            raise ValueError(f"layers of at least one output and 1 to {MOST_K} inputs are wanted")
        for t, what in ((scale, "scale"),) + (((bias, "bias"),) if bias is not None else ()):
            if t.dtype is not torch.float32 or tuple(t.shape) != (N,) or t.device != codes.device:
                raise ValueError(f"{what} must be a float32 [{N}] tensor on {codes.device}")
        width = _padded(K)
        if K != width or not codes.is_contiguous() or codes.data_ptr() % 16:
            rows = torch.zeros((N, width), dtype=torch.int8, device=codes.device)
            rows[:, :K] = codes
            codes = rows
        self.N, self.K, self.device = N, K, codes.device
        self.codes, self.scale = codes, scale.contiguous()
        self.bias = None if bias is None else bias.contiguous()
        self.clamp = clamp
        self._clamp, self._width = _clamp(clamp), width
        self._weights = (self.codes.data_ptr(), width, self.scale.data_ptr(),
                         0 if bias is None else self.bias.data_ptr(), N, K)

    def __reduce__(self):
        # a copy is made anew from the weights: its tensors lie elsewhere
        own = {k: v for k, v in self.__dict__.items() if k not in self._fixed and k not in ("_clamp", "_width", "_weights")}
        return type(self), (self.codes[:, :self.K], self.scale, self.bias, self.clamp), own or None

    @classmethod
    def from_weight(cls, weight, bias=None, clamp: Optional[float] = None):
        """A layer whose weights [N, K] (float16, bfloat16 or float32) are quantised by output channel."""
        codes, scale = quantize_rows(weight)
        return cls(codes, scale, bias=bias, clamp=clamp)

    def _output(self, T, out, out_dtype):
        """The output tensor, and its address, type and row stride."""
        if out is None:
            dt = out_dtype or _s._torch.float32
            if dt not in _s._DT:
                raise ValueError("the output must be float16, bfloat16 or float32")
            out = _s._empty(T, self.N, dtype=dt, device=self.device)
            return out, out.data_ptr(), _s._DT[dt], self.N
        if out.dim() != 2 or tuple(out.shape) != (T, self.N) or out.device != self.device or out.dtype not in _s._DT \
                or (out.stride(1) != 1 and self.N != 1) or (out_dtype or out.dtype) != out.dtype \
                or (T > 1 and out.stride(0) < self.N):
            raise ValueError(f"out must be a float16, bfloat16 or float32 [{T}, {self.N}] tensor on {self.device} with "
                             "contiguous channels and rows that do not overlap")
        return out, out.data_ptr(), _s._DT[out.dtype], out.stride(0)

    def forward(self, x, out=None, out_dtype=None):
        """x [tokens, K] float16, bfloat16 or float32 (any row stride) -> [tokens, N]: `out`, which shares no memory
        with x, or a new tensor of `out_dtype` (float32 by default)."""
        L, dev = _s._lib, self.device
        x, row = _rows2(x, self.K, dev, "x")
        T = x.shape[0]
        y, yp, yd, yr = self._output(T, out, out_dtype)
        size = L.cl_int8_work_bytes(T, self.N, self.K, 0)
        work = _s._empty(size, dtype=_s._torch.uint8, device=dev) if size else None
        st = L.cl_call(_FORWARD, _pack_forward(x.data_ptr(), _s._DT[x.dtype], row, T, self._clamp, *self._weights, yp, yd, yr,
                                               work.data_ptr() if size else 0, size, _s._stream(dev)))
        if st:
            _s._check(st, "cl_int8_forward")
        return y

    __call__ = forward

    def forward_codes(self, codes, scale, out=None, out_dtype=None):
        """The same from activations that are quantised already (quantize_rows; the layer's clamp is not applied): int8 codes
        [tokens, K] and float32 scales [tokens], for layers that share their input."""
        L, dev = _s._lib, self.device
        torch = _s._torch
        if codes.dim() != 2 or codes.dtype is not torch.int8 or codes.device != dev or codes.shape[1] != self.K:
            raise ValueError(f"codes must be an int8 [tokens, {self.K}] tensor on {dev}")
        T = codes.shape[0]
        if scale.dtype is not torch.float32 or tuple(scale.shape) != (T,) or scale.device != dev:
            raise ValueError(f"scale must be a float32 [{T}] tensor on {dev}")
        scale = scale.contiguous()
        y, yp, yd, yr = self._output(T, out, out_dtype)
        whole, row = _whole_rows(codes) if T else (True, self._width)
        if not whole:
            rows = _s._empty(T, self._width, dtype=torch.int8, device=dev)
            rows[:, :self.K] = codes
            codes, row = rows, self._width
        size = L.cl_int8_work_bytes(T, self.N, self.K, 1)
        work = _s._empty(size, dtype=_s._torch.uint8, device=dev) if size else None
        st = L.cl_call(_LINEAR, _pack_linear(codes.data_ptr(), row, scale.data_ptr(), T, *self._weights, yp, yd, yr,
                                             work.data_ptr() if size else 0, size, _s._stream(dev)))
        if st:
            _s._check(st, "cl_int8_linear")
        return y
