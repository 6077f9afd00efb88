"""What a batch of sequences needs around a paged cache, over libgemm's C ABI
(include/gemm.h).

``kv_plan``: from the sequences' lengths and new tokens, on the GPU, the row
offsets, positions, cache slots and page table entries of a step, whose pages come
off a stack of free ones.

``Rotary`` and ``rotary``: rotary positions of queries and keys, and the way back.

Arguments, streams and errors as in ``lowbit``.
"""
from __future__ import annotations

import math
from collections import namedtuple

import torch

from . import binding
from .binding import GemmError
from .lowbit import _I32, _TYPES, _empty, _Handle, _stream

LAYOUTS = ("half", "interleaved")
SCALINGS = (None, "linear", "ntk", "yarn")

Plan = namedtuple("Plan", "starts first lengths positions slots available heights")


def kv_plan(page_table, lengths, counts, free, available, page_tokens, tokens, update=False, stream=None) -> Plan:
    """The plan of a step in which sequence b, with lengths[b] tokens in the cache,
    gets counts[b] more (0: it rests).  `free` is a stack of free pages of which the
    first available[0] are on it, `tokens` (a host number) the rows of the step: the
    sum of the counts, or more (the rows behind get position and slot -1; ``rotary``
    and the calls on a cache leave such rows as they were, the latter with ERR_INDEX).

    Writes the pages that the new tokens begin into page_table and returns a Plan:
    starts and first as kv_append takes them, lengths after the step as
    kv_attention does, positions (int32) and slots (int64: page * page_tokens +
    place in it) of the rows, what is then available, and the stack's heights
    before each sequence and after the last.  With `update`, lengths and
    available are written in place (a step recorded in a graph goes on where the
    last replay ended).  Bad numbers, counts past `tokens` (sequences get what there
    is room for, in their order) and pages that run out are reported by
    ``binding.debug_status()`` as ERR_INDEX; the tokens without a page have slot -1."""
    index = page_table.get_device()
    if not (page_table.dtype is lengths.dtype is counts.dtype is free.dtype is available.dtype is _I32 and page_table.is_cuda
            and lengths.get_device() == index and counts.get_device() == index and free.get_device() == index
            and available.get_device() == index and page_table.is_contiguous() and lengths.is_contiguous()
            and counts.is_contiguous() and free.is_contiguous() and page_table.dim() == 2
            and lengths.dim() == counts.dim() == free.dim() == 1 and available.numel() == 1):
        raise TypeError("page_table (2-D), lengths, counts, free (1-D) and available (one element) must be contiguous int32 "
                        "tensors on one CUDA device")
    n, width = page_table.shape
    if lengths.shape[0] != n or counts.shape[0] != n:
        raise ValueError(f"{n} page table rows, {lengths.shape[0]} lengths and {counts.shape[0]} counts do not fit together")
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    if abs(page_tokens) >= 1 << 31:     # not one, but ctypes would take its low 32 bits
        page_tokens = 0
    device = page_table.device
    slots = _empty((tokens,), torch.int64, device, stream)
    parts = [n + 1, n + 1, n, tokens] if update else [n + 1, n + 1, n, tokens, n, 1]
    starts, heights, first, positions, *after = _empty((sum(parts),), _I32, device, stream).split_with_sizes(parts)
    new_lengths, left = (lengths, available) if update else after
    rc = binding.lib().gemm_kv_plan(page_table.data_ptr() or None, width, lengths.data_ptr() or None, counts.data_ptr() or None,
                                    free.data_ptr() or None, free.shape[0], available.data_ptr(), page_tokens, tokens, n,
                                    starts.data_ptr(), first.data_ptr() or None, new_lengths.data_ptr() or None,
                                    heights.data_ptr(), left.data_ptr(), positions.data_ptr() or None, slots.data_ptr() or None,
                                    _stream(stream, index))
    if rc:
        raise GemmError(rc, "gemm_kv_plan")
    return Plan(starts, first, new_lengths, positions, slots, left, heights)


class Rotary(_Handle):
    """The rotation of a head's first `rotary_dim` elements: pair i (elements i and
    i + rotary_dim / 2 in the layout "half", 2i and 2i + 1 in "interleaved") by
    position * f_i, f_i = base ** (-2i / rotary_dim) radians.  For contexts
    `factor` times the one that a model was trained on, `scaling` is
      "linear"  f / factor
      "ntk"     base * factor ** (rotary_dim / (rotary_dim - 2)) for base
      "yarn"    with r = original * f / (2 pi) turns in the original context
                and k = (r - 1) / 31 held to [0, 1]: k f + (1 - k) f / factor,
                and results times 0.1 ln(factor) + 1 (under 1 for a factor under 1)
    or give `frequencies` (and `magnitude`) as they are: for models whose code has its
    ramp over the pairs' numbers, or three bands of them."""

    __slots__ = ("rotary_dim", "layout", "frequencies", "magnitude", "turns", "device", "index", "_ptr", "_layout")

    def __init__(self, rotary_dim, base=10000.0, layout="half", scaling=None, factor=1.0, original=None, frequencies=None,
                 magnitude=None, device="cuda"):
        if rotary_dim < 2 or rotary_dim % 2:
            raise ValueError("rotary_dim must be even and positive")
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {LAYOUTS}")
        if scaling not in SCALINGS:
            raise ValueError(f"scaling must be one of {SCALINGS}")
        if not base > 0 or not factor > 0:
            raise ValueError("base and factor must be positive")
        half, given = rotary_dim // 2, magnitude
        magnitude = 1.0
        if frequencies is None:
            if scaling == "ntk" and rotary_dim > 2:
                base = base * factor ** (rotary_dim / (rotary_dim - 2))
            frequencies = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
            if scaling == "linear":
                frequencies = [f / factor for f in frequencies]
            if scaling == "yarn":
                if not original or original <= 0:
                    raise ValueError('scaling "yarn" needs the original context length')
                kept = [min(1.0, max(0.0, (original * f / (2 * math.pi) - 1.0) / 31.0)) for f in frequencies]
                frequencies = [k * f + (1 - k) * f / factor for k, f in zip(kept, frequencies)]
                magnitude = 0.1 * math.log(factor) + 1.0
        else:
            frequencies = [float(f) for f in frequencies]
            if scaling is not None:
                raise ValueError("frequencies are taken as they are: no scaling")
        if given is not None:
            magnitude = float(given)
        if (len(frequencies) != half or not all(math.isfinite(f) for f in frequencies)
                or not abs(magnitude) <= torch.finfo(torch.float32).max):
            raise ValueError(f"{half} finite frequencies and a finite magnitude are wanted")
        # in turns times 2^64, modulo 2^64, as signed numbers
        turns = [round(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in frequencies]
        turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        if not turns.is_cuda:
            raise TypeError("a Rotary is on a CUDA device")
        self._hold(rotary_dim=int(rotary_dim), layout=layout, frequencies=tuple(frequencies), magnitude=magnitude, turns=turns,
                   device=turns.device, index=turns.get_device(), _ptr=turns.data_ptr(), _layout=LAYOUTS.index(layout))

    def __reduce__(self):
        return _rotary_again, (self.rotary_dim, self.layout, self.frequencies, self.magnitude, str(self.device))


def _rotary_again(rotary_dim, layout, frequencies, magnitude, device):
    return Rotary(rotary_dim, layout=layout, frequencies=frequencies, magnitude=magnitude, device=device)


def _rows(t, name, kind, index, like=None):
    """(row stride, head stride) of rows x heads x dim with dense elements."""
    if t.dim() != 3 or t.get_device() != index or t.dtype is not kind or (t.stride(2) != 1 and t.shape[2] > 1):
        raise TypeError(f"{name} must be a tensor of rows x heads x dim with dense elements, of Q's type and on cuda:{index}")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(like.shape)}")
    return t.stride(0), t.stride(1)


def rotary(Q, K, positions, table: Rotary, inverse=False, out=None, stream=None):
    """Q and K (rows x heads x head_dim; float32, bfloat16 or float16; any row and
    head strides; K may be None) with every head turned by its row's position (int32,
    as kv_plan gives them), or, with `inverse`, turned back: the gradient's way.
    Returns (Q, K) anew, or in `out`, a pair that may be (Q, K) itself.  Rows with a
    negative position are not written.  Autograd does not see this call: where it
    records (not under torch.no_grad or in a Function's forward), tensors that
    require a gradient are refused."""
    kind, index = Q.dtype, table.index
    number = _TYPES.get(kind)
    if number is None:
        raise TypeError("Q must be float32, bfloat16 or float16")
    if torch.is_grad_enabled() and (Q.requires_grad or (K is not None and K.requires_grad)
                                    or (out is not None and any(t is not None and t.requires_grad for t in out))):
        raise TypeError("autograd does not see rotary: its results would have no gradient (the way back is inverse=True, of the "
                        "results' gradients)")
    qr, qh = _rows(Q, "Q", kind, index)
    rows, q_heads, dim = Q.shape
    if not (positions.dtype is _I32 and positions.get_device() == index and positions.dim() == 1 and positions.is_contiguous()):
        raise TypeError(f"positions must be a contiguous int32 tensor on {table.device}")
    if positions.shape[0] != rows:
        raise ValueError(f"{rows} rows and {positions.shape[0]} positions")
    if table.rotary_dim > dim:
        raise ValueError(f"heads of {dim} elements, of which {table.rotary_dim} are to be turned")
    if out is None:
        q_out, k_out = _empty((rows, q_heads, dim), kind, Q.device, stream), None
        qor, qoh = q_heads * dim, dim
    else:
        q_out, k_out = out
        qor, qoh = _rows(q_out, "out[0]", kind, index, Q)
    if K is None:
        k_args = (None, 0, 0, None, 0, 0, 0)
    else:
        kr, kh = _rows(K, "K", kind, index)
        k_rows, k_heads, k_dim = K.shape
        if k_rows != rows or k_dim != dim:
            raise ValueError(f"Q has {rows} rows of heads of {dim} elements, K {k_rows} of {k_dim}")
        if out is None:
            k_out = _empty((rows, k_heads, dim), kind, Q.device, stream)
            kor, koh = k_heads * dim, dim
        else:
            kor, koh = _rows(k_out, "out[1]", kind, index, K)
        k_args = (K.data_ptr() or None, kr, kh, k_out.data_ptr() or None, kor, koh, k_heads)
    rc = binding.lib().gemm_rotary(Q.data_ptr() or None, qr, qh, q_out.data_ptr() or None, qor, qoh, q_heads, *k_args, number,
                                   rows, dim, table.rotary_dim, table._layout, positions.data_ptr() or None, table._ptr,
                                   table.magnitude, inverse, _stream(stream, index))
    if rc:
        raise GemmError(rc, "gemm_rotary")
    return q_out, k_out
