"""Products with operands held in few bits, over libgemm's C ABI (include/gemm.h).

``w4_quantize`` / ``w4_dequantize`` / ``gemm_w4``: C = X W for a few rows X and
a W of 4-bit integers with a bfloat16 scale for each column and group of rows.

``KvCache`` with ``kv_append`` / ``kv_read`` / ``kv_attention``: a paged cache of
8-bit keys and values with one scale per page and head, and the attention of
ragged queries over it.

As in ``binding``: argument marshalling only, on torch's current stream unless
one is given, asynchronous, errors as ``binding.GemmError`` (a status of the
library), ``TypeError`` (a tensor's type, device or layout) or ``ValueError``
(sizes that do not fit together).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding
from .binding import GemmError

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
PAGE_TOKENS = (16, 32, 64, 128)
HEAD_DIMS = (64, 128)
GROUPS = (32, 64, 128)


class _CKvCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def _stream(stream, device):
    """The address of `stream`, or of the current stream of `device` (asked for
    by number: making a Stream object of it costs 3 us, a kernel's launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index) or None
    return stream.cuda_stream or None


def _empty(shape, dtype, device, stream):
    """An output that belongs to the stream which writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need(cond, name, what):
    if not cond:
        raise TypeError(f"{name} must be {what}")


def _rows2(t, name):
    """A 2-D CUDA tensor whose rows are dense; returns its row stride."""
    _need(t.is_cuda and t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1), name,
          "a 2-D CUDA tensor with dense rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


# ---- 4-bit weights ----------------------------------------------------------

class W4Matrix:
    """A K x N matrix in 4 bits: the packed codes (uint8), the scales
    (bfloat16), its sizes and the group length.  Layout: include/gemm.h."""

    __slots__ = ("codes", "scales", "K", "N", "group", "_args")

    def __init__(self, codes, scales, K, N, group):
        code_bytes, scale_bytes = w4_sizes(K, N, group)
        _need(codes.is_cuda and codes.is_contiguous() and codes.element_size() * codes.numel() == code_bytes,
              "codes", f"a contiguous CUDA tensor of {code_bytes} bytes")
        _need(scales.is_cuda and scales.is_contiguous() and scales.dtype == torch.bfloat16
              and 2 * scales.numel() == scale_bytes, "scales",
              f"a contiguous CUDA bfloat16 tensor of {scale_bytes // 2} elements")
        if codes.device != scales.device:
            raise TypeError("codes and scales must be on one device")
        self.codes, self.scales, self.K, self.N, self.group = codes, scales, int(K), int(N), int(group)
        self._args = (codes.data_ptr() or None, scales.data_ptr() or None)

    @property
    def device(self):
        return self.codes.device


def w4_sizes(K: int, N: int, group: int):
    """(bytes of the codes, bytes of the scales) of a K x N matrix."""
    a, b = ctypes.c_int64(), ctypes.c_int64()
    rc = binding.lib().gemm_w4_sizes(K, N, group, ctypes.byref(a), ctypes.byref(b))
    if rc != binding.OK:
        raise GemmError(rc, "gemm_w4_sizes")
    return a.value, b.value


def w4_quantize(B, group=128, stream=None) -> W4Matrix:
    """B (K x N; float32, bfloat16 or float16, dense rows) in 4 bits: for each
    column and `group` rows s = max|b| * (1 / 7) in bfloat16 and q = round(b / s)."""
    ldb = _rows2(B, "B")
    _need(B.dtype in _TYPES, "B", "float32, bfloat16 or float16")
    K, N = B.shape
    code_bytes, scale_bytes = w4_sizes(K, N, group)
    codes = _empty(code_bytes, torch.uint8, B.device, stream)
    scales = _empty(scale_bytes // 2, torch.bfloat16, B.device, stream)
    W = W4Matrix(codes, scales, K, N, group)
    rc = binding.lib().gemm_w4_quantize(B.data_ptr() or None, ldb, _TYPES[B.dtype], K, N, group, *W._args,
                                        _stream(stream, B.device))
    if rc != binding.OK:
        raise GemmError(rc, "gemm_w4_quantize")
    return W


def w4_dequantize(W: W4Matrix, out=None, dtype=torch.bfloat16, stream=None):
    """The K x N values that W stands for, each rounded once to `dtype` (or
    into `out`)."""
    if out is None:
        out = _empty((W.K, W.N), dtype, W.device, stream)
    ldb = _rows2(out, "out")
    _need(out.dtype in _TYPES, "out", "float32, bfloat16 or float16")
    _same_device("out", out, W.device)
    if tuple(out.shape) != (W.K, W.N):
        raise ValueError(f"out has shape {tuple(out.shape)}, not {(W.K, W.N)}")
    rc = binding.lib().gemm_w4_dequantize(*W._args, W.K, W.N, W.group, out.data_ptr() or None, ldb,
                                          _TYPES[out.dtype], _stream(stream, out.device))
    if rc != binding.OK:
        raise GemmError(rc, "gemm_w4_dequantize")
    return out


def _same_device(name, t, device):
    if t.device != device:
        raise TypeError(f"{name} is on {t.device}, not on {device}")


def gemm_w4(X, W: W4Matrix, C=None, dtype=None, stream=None):
    """C = X W.  X: M x K, bfloat16 or float16, dense rows; C: M x N of X's
    type or float32 (`dtype`, or `C` itself); X's type by default.  Returns C."""
    ldx = _rows2(X, "X")
    xt = X.dtype
    _need(xt == torch.bfloat16 or xt == torch.float16, "X", "bfloat16 or float16")
    M, K = X.shape
    if K != W.K:
        raise ValueError(f"X has {K} columns, W has {W.K} rows")
    _same_device("X", X, W.codes.device)
    if C is None:
        C = _empty((M, W.N), dtype or xt, X.device, stream)
        ldc = W.N
    else:
        ldc = _rows2(C, "C")
        _same_device("C", C, X.device)
        if tuple(C.shape) != (M, W.N):
            raise ValueError(f"C has shape {tuple(C.shape)}, not {(M, W.N)}")
    _need(C.dtype == xt or C.dtype == torch.float32, "C", "of X's type or float32")
    rc = binding.lib().gemm_w4(X.data_ptr() or None, ldx, _TYPES[xt], *W._args, C.data_ptr() or None, ldc,
                               _TYPES[C.dtype], M, K, W.N, W.group, _stream(stream, X.device))
    if rc != binding.OK:
        raise GemmError(rc, "gemm_w4")
    return C


# ---- the 8-bit cache -----------------------------------------------------------

class KvCache:
    """A paged cache of keys and values: codes uint8 [pages, heads,
    page_tokens, head_dim] and scales float32 [pages, heads] of each."""

    __slots__ = ("k_codes", "v_codes", "k_scales", "v_scales", "heads", "head_dim", "page_tokens", "device",
                 "_c", "_ref")

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        shape = tuple(k_codes.shape)
        _need(len(shape) == 4 and shape[2] in PAGE_TOKENS and shape[3] in HEAD_DIMS, "k_codes",
              f"[pages, heads, page_tokens in {PAGE_TOKENS}, head_dim in {HEAD_DIMS}]")
        for name, t, want, dt in (("k_codes", k_codes, shape, torch.uint8), ("v_codes", v_codes, shape, torch.uint8),
                                  ("k_scales", k_scales, shape[:2], torch.float32),
                                  ("v_scales", v_scales, shape[:2], torch.float32)):
            _need(tuple(t.shape) == want and t.dtype == dt and t.is_cuda and t.is_contiguous()
                  and t.device == k_codes.device, name, f"a contiguous CUDA {dt} tensor of shape {want}")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.device = k_codes.device
        pages, self.heads, self.page_tokens, self.head_dim = shape
        self._c = _CKvCache(k_codes.data_ptr() or None, v_codes.data_ptr() or None, k_scales.data_ptr() or None,
                            v_scales.data_ptr() or None, pages, self.heads, self.page_tokens, self.head_dim)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, pages, heads, head_dim, page_tokens=64, device="cuda"):
        """A cache of `pages` pages; a page needs no initial contents."""
        shape = (pages, heads, page_tokens, head_dim)
        return cls(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))


def _batch(cache, page_table, starts, at, name):
    """Checks the index tensors of a call; returns (table width, sequences)."""
    for n, t, dims in (("page_table", page_table, 2), ("starts", starts, 1), (name, at, 1)):
        if t.dtype != torch.int32 or t.dim() != dims or t.device != cache.device or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous {dims}-D int32 tensor on {cache.device}")
    sequences = at.shape[0]
    if page_table.shape[0] != sequences or starts.shape[0] != sequences + 1:
        raise ValueError(f"{sequences} entries of {name}, {page_table.shape[0]} page table rows and "
                         f"{starts.shape[0]} starts do not fit together")
    return page_table.shape[1], sequences


def _rows3(t, name, cache, heads=None):
    """Rows of heads x head_dim elements with dense elements; returns (row stride, head stride)."""
    if (t.dim() != 3 or t.device != cache.device or t.shape[2] != cache.head_dim or t.stride(2) != 1
            or (heads is not None and t.shape[1] != heads)):
        raise TypeError(f"{name} must be a tensor on {cache.device} of rows x {heads or 'heads'} x "
                        f"{cache.head_dim} with dense elements")
    return t.stride(0), t.stride(1)


def kv_append(cache: KvCache, K, V, page_table, starts, first, stream=None):
    """Writes new keys and values (tokens x heads x head_dim; float32, bfloat16
    or float16; any row and head strides) into the cache: row starts[b] + i
    becomes token first[b] + i of sequence b.  A page's scale grows to the
    largest magnitude / 127, and its older codes with it."""
    width, sequences = _batch(cache, page_table, starts, first, "first")
    kr, kh = _rows3(K, "K", cache, cache.heads)
    vr, vh = _rows3(V, "V", cache, cache.heads)
    _need(K.dtype in _TYPES and V.dtype == K.dtype, "K and V", "of one type: float32, bfloat16 or float16")
    if K.shape[0] != V.shape[0]:
        raise ValueError(f"{K.shape[0]} keys and {V.shape[0]} values")
    rc = binding.lib().gemm_kv_append(cache._ref, K.data_ptr() or None, kr, kh, V.data_ptr() or None, vr, vh,
                                      _TYPES[K.dtype], page_table.data_ptr() or None, width, starts.data_ptr(),
                                      first.data_ptr() or None, K.shape[0], sequences, _stream(stream, cache.device))
    if rc != binding.OK:
        raise GemmError(rc, "gemm_kv_append")


def kv_read(cache: KvCache, page_table, starts, first, tokens, dtype=torch.bfloat16, stream=None):
    """(K, V) read back, each tokens x heads x head_dim of `dtype`: row
    starts[b] + i is token first[b] + i of sequence b.  `tokens` is starts[-1],
    known on the host."""
    width, sequences = _batch(cache, page_table, starts, first, "first")
    _need(dtype in _TYPES, "dtype", "float32, bfloat16 or float16")
    K = _empty((tokens, cache.heads, cache.head_dim), dtype, cache.device, stream)
    V = _empty((tokens, cache.heads, cache.head_dim), dtype, cache.device, stream)
    rc = binding.lib().gemm_kv_read(cache._ref, K.data_ptr() or None, V.data_ptr() or None, _TYPES[dtype],
                                    page_table.data_ptr() or None, width, starts.data_ptr(),
                                    first.data_ptr() or None, tokens, sequences, _stream(stream, cache.device))
    if rc != binding.OK:
        raise GemmError(rc, "gemm_kv_read")
    return K, V


def kv_attention(Q, cache: KvCache, page_table, starts, lengths, scale=None, causal=True, window=0, out=None,
                 stream=None):
    """Attention of Q (tokens x q_heads x head_dim; bfloat16 or float16) over
    the cache.  Sequence b has lengths[b] tokens and the queries starts[b] ..
    starts[b + 1] - 1, which stand at its last positions; with `causal` a query
    sees the tokens up to its own, with `window` > 0 the last `window` of
    them.  scale: 1 / sqrt(head_dim) by default.  A query that sees nothing
    gets 0.  Returns O, shaped and typed like Q."""
    width, sequences = _batch(cache, page_table, starts, lengths, "lengths")
    qr, qh = _rows3(Q, "Q", cache)
    _need(Q.dtype == torch.bfloat16 or Q.dtype == torch.float16, "Q", "bfloat16 or float16")
    if out is None:
        out = _empty(Q.shape, Q.dtype, Q.device, stream)
    else:
        _need(out.dtype == Q.dtype and out.shape == Q.shape, "out", "of Q's type and shape")
    orow, oh = _rows3(out, "out", cache)
    if scale is None:
        scale = 1.0 / math.sqrt(cache.head_dim)
    rc = binding.lib().gemm_kv_attention(cache._ref, Q.data_ptr() or None, qr, qh, out.data_ptr() or None, orow, oh,
                                         _TYPES[Q.dtype], Q.shape[1], scale, causal, window,
                                         page_table.data_ptr() or None, width, starts.data_ptr(),
                                         lengths.data_ptr() or None, Q.shape[0], sequences, _stream(stream, cache.device))
    if rc != binding.OK:
        raise GemmError(rc, "gemm_kv_attention")
    return out
