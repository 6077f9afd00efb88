"""Plain numpy implementations of the low-bit operators' definitions, in 64
bits except where a rule fixes a binary32 step (the quantisers), for the tests."""
from __future__ import annotations

import numpy as np

TINY = 2.0 ** -126
U = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}     # unit roundoffs


def rounding(y, kind):
    """How far a value y is from its rounding to the type, at most: u * |y|, or
    half of binary16's smallest spacing, 2^-24, where y is below 2^-14."""
    return np.maximum(U[kind] * np.abs(y), 2.0 ** -25 if kind == "fp16" else 0.0)


def bf16_round(x):
    """float32 values rounded to bfloat16 (nearest, ties to even), as float32."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    out = r.astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), out)


# ---- 4-bit weights --------------------------------------------------------------

def w4_quantize(B, group):
    """(q int8 [K, N], s float32 [groups, N]) of float32 values B."""
    B = np.asarray(B, np.float32)
    K, N = B.shape
    groups = -(-K // group)
    q, s = np.zeros((K, N), np.int8), np.zeros((groups, N), np.float32)
    for g in range(groups):
        part = B[g * group:(g + 1) * group]
        top = np.abs(part).max(0)
        bad = ~np.isfinite(part).all(0)
        with np.errstate(all="ignore"):
            sg = bf16_round((np.where(bad, 0, top) * (np.float32(1) / np.float32(7))).astype(np.float32))
            sg = np.where(sg < TINY, np.float32(0), sg)
            qg = np.clip(np.rint((part / sg).astype(np.float32)), -7, 7)
        q[g * group:(g + 1) * group] = np.where((sg == 0) | bad, 0, np.nan_to_num(qg)).astype(np.int8)
        s[g] = np.where(bad, np.float32(np.nan), sg)
    return q, s


def w4_pack(q, s, group):
    """The packed layout, element by element as the header's text gives it."""
    K, N = q.shape
    nb, kb, groups = -(-N // 16), -(-K // 64), -(-K // group)
    words = np.full(nb * kb * 128, 0x88888888, np.uint32)
    k, n = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
    at = ((n // 16) * kb + k // 64) * 128 + 4 * (4 * (n % 8) + k % 32 // 8) + 2 * (k % 64 // 32) + k % 8 // 4
    shift = 4 * (4 * (k % 2) + 2 * (k % 4 // 2) + n % 16 // 8)
    np.bitwise_xor.at(words, at.ravel(), ((((q.astype(np.int64) + 8) ^ 8) << shift).astype(np.uint32)).ravel())
    scales = np.zeros(nb * groups * 16, np.float32)
    g, n = np.meshgrid(np.arange(groups), np.arange(N), indexing="ij")
    scales[(((n // 16) * groups + g) * 8 + n % 8) * 2 + n % 16 // 8] = s
    return words, scales


def w4_values(q, s, group):
    return q.astype(np.float64) * np.repeat(s, group, 0)[:q.shape[0]].astype(np.float64)


# ---- the 8-bit cache ---------------------------------------------------------------

class Cache:
    """One operand (keys or values) of a paged cache: codes c as integers and
    float32 scales, with the append rule step by step in binary32."""

    def __init__(self, codes_u8, scales, page):
        self.c = codes_u8.astype(np.int64) - 128
        self.s = scales.astype(np.float32).copy()
        self.page = page

    def append(self, x, table, starts, first):
        x = np.asarray(x, np.float32)
        f32 = np.float32
        for b in range(len(first)):
            T = starts[b + 1] - starts[b]
            for blk in range(first[b] // self.page, -(-(first[b] + T) // self.page) if T else 0):
                lo = blk * self.page
                if lo + self.page <= first[b]:
                    continue
                begin, end = max(first[b] - lo, 0), min(first[b] + T - lo, self.page)
                p = table[b, blk]
                new = x[starts[b] + lo + begin - first[b]: starts[b] + lo + end - first[b]]      # token, head, dim
                for h in range(x.shape[1]):
                    v, old = new[:, h], self.c[p, h, :begin]
                    before = self.s[p, h] if begin else f32(0)
                    if not np.isfinite(v).all() or np.isnan(before):
                        self.c[p, h, begin:end] = 0
                        self.s[p, h] = np.nan
                        continue
                    s = max(before, f32(np.abs(v).max()) * (f32(1) / f32(127)))
                    inv = f32(1) / s if s >= TINY else f32(0)
                    self.c[p, h, begin:end] = np.clip(np.rint(v * inv), -127, 127).astype(np.int64)
                    if before < s:
                        self.c[p, h, :begin] = np.rint(old.astype(f32) * (before * inv)).astype(np.int64)
                    self.s[p, h] = s

    def tokens(self, table_row, n):
        """[heads, n, dim] values in 64 bits."""
        pages = table_row[: -(-n // self.page)]
        v = self.c[pages].astype(np.float64) * self.s[pages][..., None, None].astype(np.float64)
        return v.transpose(1, 0, 2, 3).reshape(self.c.shape[1], -1, self.c.shape[3])[:, :n]


def attention(q, k, v, table, starts, lengths, scale, causal, window):
    """(o, spread, reach): o in 64 bits and, for the tolerance, of each row
    sum_j p_j |v_j| (with the part that binary16 weights below its smallest
    spacing can add) and the largest scale * sum_d |q_d k_d|."""
    q = q.astype(np.float64)
    o = np.zeros_like(q)
    spread, reach = np.zeros_like(q), np.zeros(q.shape[:2])
    share = q.shape[1] // k.c.shape[1]
    for b in range(len(lengths)):
        n, T = lengths[b], starts[b + 1] - starts[b]
        if n == 0 or T == 0:
            continue
        kk, vv = k.tokens(table[b], n), v.tokens(table[b], n)
        # a weight of at most 2^15 times its page's share of the largest value
        # scale is off by 2^-25 at least: times 2^11 here, as spread's factor is 2^-11
        least = 2.0 ** (-25 - 15 + 11) * 127 * float(v.s[table[b, : -(-n // v.page)]].max())
        for i in range(T):
            pos = n - T + i
            if pos < 0:
                continue
            hi = pos + 1 if causal else n
            lo = max(0, pos - window + 1) if window else 0
            for h in range(q.shape[1]):
                x = q[starts[b] + i, h]
                kv, val = kk[h // share, lo:hi], vv[h // share, lo:hi]
                sc = scale * (kv @ x)
                p = np.exp(sc - sc.max())
                p /= p.sum()
                o[starts[b] + i, h] = p @ val
                spread[starts[b] + i, h] = p @ np.abs(val) + least * (hi - lo)
                reach[starts[b] + i, h] = abs(scale) * (np.abs(kv) @ np.abs(x)).max()
    return o, spread, reach


def attention_limit(o, spread, reach, dim, kind):
    """|got - o| at most: a score's binary32 error (dim + 8 roundings of at
    most reach, and a bfloat16 query's part below 2^-25 of its row's largest)
    moves a weight by as much relatively, twice for the weight and the sum;
    the weight's binary16 rounding 2^-11; exp2 and the sums 2^-18; the
    result's own rounding."""
    score = reach * (dim + 8) * 2.0 ** -23 + reach * 2.0 ** -18 * (kind == "bf16")
    return spread * (2.0 ** -11 + 2.0 ** -18 + 2 * score[..., None]) + rounding(o, kind) + 1e-30
