"""Products with operands held in few bits, over libgemm's C ABI (include/gemm.h).

``w4_quantize`` / ``w4_dequantize`` / ``gemm_w4``: C = X W for a few rows X and
a W of 4-bit integers with a bfloat16 scale for each column and group of rows.

``KvCache`` with ``kv_append`` / ``kv_read`` / ``kv_attention``: a paged cache of
8-bit keys and values with one scale per page and head, and the attention of
ragged queries over it; ``Kv4Cache`` with the same calls: one of 4 bits with a
scale per token and head.

As in ``binding``: argument marshalling only, on the current CUDA device, whose
tensors the operands have to be, and on torch's current stream unless one is
given, asynchronous, errors as ``binding.GemmError`` (a status of the library),
``TypeError`` (a tensor's type, device or layout) or ``ValueError`` (sizes that
do not fit together).
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import GemmError

_F32, _BF16, _F16, _I32 = torch.float32, torch.bfloat16, torch.float16, torch.int32
_TYPES = {_F32: 0, _BF16: 1, _F16: 2}
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
PAGE_TOKENS = (16, 32, 64, 128)
HEAD_DIMS = (64, 128)
GROUPS = (32, 64, 128)

# A small call's time is the host's: the checks below are written out in each
# function, in the fewest steps, and what is wrong is told apart only then.


class _CKv4Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _CKvCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def _empty(shape, dtype, device, stream):
    """An output that belongs to the stream which writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _stream(stream, index):
    """The address of `stream`, or of the current stream of device `index`
    (asked for by number: making a Stream object of it costs 3 us).  The
    library works on the current device, so that has to be the tensors'."""
    if _current_device() != index:
        raise TypeError(f"the tensors are on cuda:{index}, the current device is cuda:{_current_device()}")
    return (_raw_stream(index) if stream is None else stream.cuda_stream) or None


def _need(cond, name, what):
    if not cond:
        raise TypeError(f"{name} must be {what}")


def _rows2(t, name):
    """A 2-D CUDA tensor whose rows are dense; returns its row stride."""
    if not t.is_cuda or t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise TypeError(f"{name} must be a 2-D CUDA tensor with dense rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


class _Handle:
    """What holds addresses and sizes of its tensors: fixed once it is made
    (the tensors' contents are the caller's); a copy is made of tensors anew."""

    __slots__ = ()

    def _hold(self, **fields):
        for name, value in fields.items():
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__} cannot be changed: make another")

    def __delattr__(self, name):
        raise AttributeError(f"{type(self).__name__} cannot be changed: make another")


# ---- 4-bit weights ----------------------------------------------------------

class _W4Fields:
    """A W4Matrix in the making: an object of this class can be assigned to."""
    __slots__ = ("_codes", "_scales", "K", "N", "group", "index", "device", "_code_ptr", "_scale_ptr")


class W4Matrix(_Handle, _W4Fields):
    """A K x N matrix in 4 bits: the packed codes (uint8), the scales
    (bfloat16), its sizes and the group length.  Layout: include/gemm.h."""

    __slots__ = ()

    def __init__(self, codes, scales, K, N, group):
        code_bytes, scale_bytes = w4_sizes(K, N, group)
        _need(codes.is_cuda and codes.is_contiguous() and codes.element_size() * codes.numel() == code_bytes,
              "codes", f"a contiguous CUDA tensor of {code_bytes} bytes")
        _need(scales.is_cuda and scales.is_contiguous() and scales.dtype == _BF16
              and 2 * scales.numel() == scale_bytes, "scales",
              f"a contiguous CUDA bfloat16 tensor of {scale_bytes // 2} elements")
        if codes.device != scales.device:
            raise TypeError("codes and scales must be on one device")
        self._hold(_codes=codes, _scales=scales, K=int(K), N=int(N), group=int(group), index=codes.get_device(),
                   device=codes.device, _code_ptr=codes.data_ptr() or None, _scale_ptr=scales.data_ptr() or None)

    @staticmethod
    def _in(both, code_bytes, K, N, group):
        """Codes and scales one after the other in the bytes of `both`."""
        W = _W4Fields()
        W._codes, W._scales, W.K, W.N, W.group = both, code_bytes, K, N, group
        W.index, W.device = both.get_device(), both.device
        at = both.data_ptr()
        W._code_ptr, W._scale_ptr = at or None, at + code_bytes if at else None
        W.__class__ = W4Matrix      # fixed from here on, at a fifth of what _hold takes
        return W

    def __reduce__(self):
        return type(self), (self.codes, self.scales, self.K, self.N, self.group)

    @property
    def codes(self):
        return self._codes[:self._scales] if isinstance(self._scales, int) else self._codes

    @property
    def scales(self):
        return self._codes[self._scales:].view(_BF16) if isinstance(self._scales, int) else self._scales


def w4_sizes(K: int, N: int, group: int):
    """(bytes of the codes, bytes of the scales) of a K x N matrix."""
    if group not in GROUPS or K < 0 or N < 0:
        raise GemmError(binding.ERR_INVALID_ARG, "gemm_w4_sizes")
    blocks = -(-N // 16)
    return blocks * -(-K // 64) * 512, blocks * -(-K // group) * 32


def w4_quantize(B, group=128, stream=None) -> W4Matrix:
    """B (K x N; float32, bfloat16 or float16, dense rows) in 4 bits: for each
    column and `group` rows s = max|b| * (1 / 7) in bfloat16 and q = round(b / s)."""
    ldb = _rows2(B, "B")
    kind = _TYPES.get(B.dtype)
    if kind is None:
        raise TypeError("B must be float32, bfloat16 or float16")
    K, N = B.shape
    code_bytes, scale_bytes = w4_sizes(K, N, group)
    W = W4Matrix._in(_empty(code_bytes + scale_bytes, torch.uint8, B.device, stream), code_bytes, K, N, group)
    rc = binding.lib().gemm_w4_quantize(B.data_ptr() or None, ldb, kind, K, N, group, W._code_ptr, W._scale_ptr,
                                        _stream(stream, W.index))
    if rc:
        raise GemmError(rc, "gemm_w4_quantize")
    return W


def w4_dequantize(W: W4Matrix, out=None, dtype=torch.bfloat16, stream=None):
    """The K x N values that W stands for, each rounded once to `dtype` (or
    into `out`)."""
    K, N = W.K, W.N
    if out is None:
        out = _empty((K, N), dtype, W.device, stream)
        ldb = N
    else:
        ldb, dtype = _rows2(out, "out"), out.dtype
        _need(out.get_device() == W.index, "out", f"on {W.device}")
        if tuple(out.shape) != (K, N):
            raise ValueError(f"out has shape {tuple(out.shape)}, not {(K, N)}")
    kind = _TYPES.get(dtype)
    if kind is None:
        raise TypeError("out must be float32, bfloat16 or float16")
    rc = binding.lib().gemm_w4_dequantize(W._code_ptr, W._scale_ptr, K, N, W.group, out.data_ptr() or None, ldb, kind,
                                          _stream(stream, W.index))
    if rc:
        raise GemmError(rc, "gemm_w4_dequantize")
    return out


def gemm_w4(X, W: W4Matrix, C=None, dtype=None, stream=None):
    """C = X W.  X: M x K, bfloat16 or float16, dense rows; C: M x N of X's
    type or float32 (`dtype`, or `C` itself); X's type by default.  Returns C."""
    ldx = _rows2(X, "X")
    xt = X.dtype
    if xt is not _BF16 and xt is not _F16:
        raise TypeError("X must be bfloat16 or float16")
    M, K = X.shape
    N, index = W.N, W.index
    if K != W.K:
        raise ValueError(f"X has {K} columns, W has {W.K} rows")
    if X.get_device() != index:
        raise TypeError(f"X is on {X.device}, not on {W.device}")
    if C is None:
        ct = dtype or xt
        C = _empty((M, N), ct, X.device, stream)
        ldc = N
    else:
        ldc, ct = _rows2(C, "C"), C.dtype
        _need(C.get_device() == index, "C", f"on {W.device}")
        if tuple(C.shape) != (M, N):
            raise ValueError(f"C has shape {tuple(C.shape)}, not {(M, N)}")
    if ct is not xt and ct is not _F32:
        raise TypeError("C must be of X's type or float32")
    rc = binding.lib().gemm_w4(X.data_ptr() or None, ldx, _TYPES[xt], W._code_ptr, W._scale_ptr, C.data_ptr() or None, ldc,
                               _TYPES[ct], M, K, N, W.group, _stream(stream, index))
    if rc:
        raise GemmError(rc, "gemm_w4")
    return C


# ---- the caches ------------------------------------------------------------------

class KvCache(_Handle):
    """A paged cache of keys and values in 8 bits: codes uint8 [pages, heads,
    page_tokens, head_dim] and scales float32 [pages, heads] of each."""

    __slots__ = ("k_codes", "v_codes", "k_scales", "v_scales", "heads", "head_dim", "page_tokens", "device", "index",
                 "_c", "_ref")
    _append, _read, _attention = "gemm_kv_append", "gemm_kv_read", "gemm_kv_attention"

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        shape = tuple(k_codes.shape)
        _need(len(shape) == 4 and shape[2] in PAGE_TOKENS and shape[3] in HEAD_DIMS, "k_codes",
              f"[pages, heads, page_tokens in {PAGE_TOKENS}, head_dim in {HEAD_DIMS}]")
        for name, t, want, dt in (("k_codes", k_codes, shape, torch.uint8), ("v_codes", v_codes, shape, torch.uint8),
                                  ("k_scales", k_scales, shape[:2], _F32), ("v_scales", v_scales, shape[:2], _F32)):
            _need(tuple(t.shape) == want and t.dtype == dt and t.is_cuda and t.is_contiguous()
                  and t.device == k_codes.device, name, f"a contiguous CUDA {dt} tensor of shape {want}")
        pages, heads, page_tokens, head_dim = shape
        c = _CKvCache(k_codes.data_ptr() or None, v_codes.data_ptr() or None, k_scales.data_ptr() or None,
                      v_scales.data_ptr() or None, pages, heads, page_tokens, head_dim)
        self._hold(k_codes=k_codes, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales, device=k_codes.device,
                   index=k_codes.get_device(), heads=heads, page_tokens=page_tokens, head_dim=head_dim, _c=c,
                   _ref=ctypes.byref(c))

    def __reduce__(self):
        return type(self), (self.k_codes, self.v_codes, self.k_scales, self.v_scales)

    @classmethod
    def empty(cls, pages, heads, head_dim, page_tokens=64, device="cuda"):
        """A cache of `pages` pages; a page needs no initial contents."""
        shape = (pages, heads, page_tokens, head_dim)
        return cls(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.zeros(shape[:2], dtype=_F32, device=device) for _ in range(2)))


class Kv4Cache(_Handle):
    """A paged cache of keys and values in 4 bits, with a scale for each token
    and head of either: uint8 [pages, heads, page_tokens * (head_dim + 4)], which
    holds for a page and head the codes of keys and of values and their bfloat16
    scales.  Layout: include/gemm.h."""

    __slots__ = ("data", "heads", "head_dim", "page_tokens", "device", "index", "_c", "_ref")
    _append, _read, _attention = "gemm_kv4_append", "gemm_kv4_read", "gemm_kv4_attention"

    def __init__(self, data, page_tokens, head_dim):
        _need(page_tokens in PAGE_TOKENS, "page_tokens", f"one of {PAGE_TOKENS}")
        _need(head_dim in HEAD_DIMS, "head_dim", f"one of {HEAD_DIMS}")
        record = page_tokens * (head_dim + 4)
        _need(data.dim() == 3 and data.shape[2] == record and data.dtype == torch.uint8 and data.is_cuda
              and data.is_contiguous(), "data", f"a contiguous CUDA uint8 tensor [pages, heads, {record}]")
        pages, heads, _ = data.shape
        c = _CKv4Cache(data.data_ptr() or None, pages, heads, page_tokens, head_dim)
        self._hold(data=data, device=data.device, index=data.get_device(), heads=heads, page_tokens=int(page_tokens),
                   head_dim=int(head_dim), _c=c, _ref=ctypes.byref(c))

    def __reduce__(self):
        return type(self), (self.data, self.page_tokens, self.head_dim)

    @classmethod
    def empty(cls, pages, heads, head_dim, page_tokens=64, device="cuda"):
        """A cache of `pages` pages; a page needs no initial contents."""
        return cls(torch.empty((pages, heads, page_tokens * (head_dim + 4)), dtype=torch.uint8, device=device),
                   page_tokens, head_dim)


def _batch(cache, page_table, starts, at, name):
    """Checks the index tensors of a call; returns (table width, sequences)."""
    index = cache.index
    if not (page_table.dtype is starts.dtype is at.dtype is _I32 and page_table.get_device() == index
            and starts.get_device() == index and at.get_device() == index and page_table.is_contiguous()
            and starts.is_contiguous() and at.is_contiguous() and page_table.dim() == 2 and starts.dim() == at.dim() == 1):
        raise TypeError(f"page_table (2-D), starts and {name} (1-D) must be contiguous int32 tensors on {cache.device}")
    rows, width = page_table.shape
    sequences = at.shape[0]
    if rows != sequences or starts.shape[0] != sequences + 1:
        raise ValueError(f"{sequences} entries of {name}, {rows} page table rows and {starts.shape[0]} starts do not "
                         "fit together")
    return width, sequences


def _rows3(t, name, cache):
    """Rows of heads x head_dim elements with dense elements; returns (rows, heads, row stride, head stride)."""
    if t.dim() == 3 and t.get_device() == cache.index:
        rows, heads, dim = t.shape
        row, head, one = t.stride()
        if dim == cache.head_dim and one == 1:
            return rows, heads, row, head
    raise TypeError(f"{name} must be a tensor on {cache.device} of rows x heads x {cache.head_dim} with dense elements")


def kv_append(cache, K, V, page_table, starts, first, stream=None):
    """Writes new keys and values (tokens x heads x head_dim; float32, bfloat16
    or float16; any row and head strides) into a KvCache or Kv4Cache: row
    starts[b] + i becomes token first[b] + i of sequence b.  In 8 bits a page's
    scale grows to the largest magnitude / 127, and its older codes with it; in 4
    bits each token and head gets a scale of its own, the largest magnitude / 7."""
    width, sequences = _batch(cache, page_table, starts, first, "first")
    rows, heads, kr, kh = _rows3(K, "K", cache)
    v_rows, v_heads, vr, vh = _rows3(V, "V", cache)
    kind = _TYPES.get(K.dtype)
    if kind is None or V.dtype is not K.dtype:
        raise TypeError("K and V must be of one type: float32, bfloat16 or float16")
    if heads != cache.heads or v_heads != heads:
        raise TypeError(f"K and V must have {cache.heads} heads")
    if rows != v_rows:
        raise ValueError(f"{rows} keys and {v_rows} values")
    call = getattr(binding.lib(), cache._append)
    rc = call(cache._ref, K.data_ptr() or None, kr, kh, V.data_ptr() or None, vr, vh, kind,
              page_table.data_ptr() or None, width, starts.data_ptr(),
              first.data_ptr() or None, rows, sequences, _stream(stream, cache.index))
    if rc:
        raise GemmError(rc, cache._append)


def kv_read(cache, page_table, starts, first, tokens, dtype=torch.bfloat16, stream=None):
    """(K, V) of a KvCache or Kv4Cache read back, each tokens x heads x head_dim of `dtype`: row
    starts[b] + i is token first[b] + i of sequence b.  `tokens` is starts[-1],
    known on the host."""
    width, sequences = _batch(cache, page_table, starts, first, "first")
    kind = _TYPES.get(dtype)
    if kind is None:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    shape = (tokens, cache.heads, cache.head_dim)
    K = _empty(shape, dtype, cache.device, stream)
    V = _empty(shape, dtype, cache.device, stream)
    call = getattr(binding.lib(), cache._read)
    rc = call(cache._ref, K.data_ptr() or None, V.data_ptr() or None, kind,
              page_table.data_ptr() or None, width, starts.data_ptr(),
              first.data_ptr() or None, tokens, sequences, _stream(stream, cache.index))
    if rc:
        raise GemmError(rc, cache._read)
    return K, V


def kv_attention(Q, cache, page_table, starts, lengths, scale=None, causal=True, window=0, out=None,
                 stream=None):
    """Attention of Q (tokens x q_heads x head_dim; bfloat16 or float16) over
    a KvCache or Kv4Cache.  Sequence b has lengths[b] tokens and the queries starts[b] ..
    starts[b + 1] - 1, which stand at its last positions; with `causal` a query
    sees the tokens up to its own, with `window` > 0 the last `window` of
    them (pages wholly before every window need not be in the table).  scale:
    1 / sqrt(head_dim) by default.  A query that sees nothing gets 0.  Returns
    O, shaped and typed like Q."""
    width, sequences = _batch(cache, page_table, starts, lengths, "lengths")
    rows, heads, qr, qh = _rows3(Q, "Q", cache)
    kind = Q.dtype
    if kind is not _BF16 and kind is not _F16:
        raise TypeError("Q must be bfloat16 or float16")
    if out is None:
        dim = cache.head_dim
        out = _empty((rows, heads, dim), kind, cache.device, stream)
        orow, oh = heads * dim, dim
    else:
        o_rows, o_heads, orow, oh = _rows3(out, "out", cache)
        _need(out.dtype is kind and o_rows == rows and o_heads == heads, "out", "of Q's type and shape")
    if scale is None:
        scale = cache.head_dim ** -0.5
    if window >= 1 << 63:       # as good as none, but ctypes would take its low 64 bits
        window = (1 << 63) - 1
    call = getattr(binding.lib(), cache._attention)
    rc = call(cache._ref, Q.data_ptr() or None, qr, qh, out.data_ptr() or None, orow, oh,
              _TYPES[kind], heads, scale, causal, window, page_table.data_ptr() or None,
              width, starts.data_ptr(), lengths.data_ptr() or None, rows, sequences,
              _stream(stream, cache.index))
    if rc:
        raise GemmError(rc, cache._attention)
    return out
