"""Attention over the paged 8-bit cache in 64 bits, with a limit on each row's
error that follows from what that row sees, and nothing else."""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}           # unit roundoffs
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}     # half of the smallest spacing


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


class Paged:
    """A cache of random codes with scales of about 0.02 (`k_scales`,
    `v_scales` may be written over, `gpu` is made of them) and a page table in a
    shuffled order."""

    def __init__(self, batch, width, heads, dim, page, seed=0, spare=3):
        from accelerator_gb300 import lowbit
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        pages, self.page, self.heads, self.dim = batch * width + spare, page, heads, dim
        shape = (pages, heads, page, dim)
        self.k, self.v = (self.normal(*shape).mul_(32).round_().clamp_(-127, 127).add_(128).to(torch.uint8) for _ in range(2))
        self.ks, self.vs = (self.normal(*shape[:2]).exp_().mul_(0.02) for _ in range(2))
        self.table = torch.randperm(pages, generator=self.g, device="cuda")[:batch * width].view(batch, width).to(torch.int32)
        self.cache = lowbit.KvCache(self.k, self.v, self.ks, self.vs)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def queries(self, rows, heads, kind, spread=1.5):
        return (self.normal(rows, heads, self.dim) * spread).to(kind)

    def page_of(self, b, i):
        return int(self.table[b, i])

    def attend(self, Q, counts, lengths, **kw):
        from accelerator_gb300 import lowbit
        return lowbit.kv_attention(Q, self.cache, self.table, ints(offsets(counts)), ints(lengths), **kw)


def attention(p, Q, counts, lengths, scale=None, causal=True, window=0):
    """(o, limit) of the rows of Q over the Paged p, in 64 bits.  The limit on
    |got - o| of a row, over the n tokens j that it sees with normalised
    weights w_j and values v_j:
      scores     a score's binary32 error is at most dim + 8 roundings of 2^-23 of
                 its largest sum of magnitudes, and a bfloat16 query's elements
                 under 2^-14 of the row's largest lose 2^-25 of that largest each (2^-18
                 over the sum); it moves a weight by as much, and their sum
      weights    w_j * (page's scale) is rounded to binary16: by 2^-11 of itself,
                 or by 2^-25 where it is 2^15 for the row's largest of them, times
                 a code of at most 127
      the rest   exp2, logarithms of scales (four roundings of numbers under 2^7)
                 and the sums: under 2^-15
      result     one rounding to Q's type, and binary32's smallest numbers."""
    scale = p.dim ** -0.5 if scale is None else scale
    o = torch.zeros(Q.shape, dtype=torch.float64, device="cuda")
    limit = torch.full_like(o, 2.0 ** -140)
    at, share, x = 0, Q.shape[1] // p.heads, Q.double()
    for b, (T, n) in enumerate(zip(counts, lengths)):
        rows, at = slice(at, at + T), at + T
        if T == 0 or n == 0:
            continue
        pages = p.table[b, : -(-n // p.page)].long()

        def dense(codes, scales):                                     # head, token, dim; head, token
            c = (codes[pages].double() - 128).transpose(0, 1).reshape(p.heads, -1, p.dim)[:, :n]
            s = scales[pages].double().t().repeat_interleave(p.page, 1)[:, :n]
            return c * s[..., None], s

        (k, _), (v, vs) = dense(p.k, p.ks), dense(p.v, p.vs)
        i = torch.arange(T, device="cuda")[:, None] + (n - T)
        j = torch.arange(n, device="cuda")[None]
        seen = (i >= 0) & ((j <= i) if causal else (j >= 0))
        if window:
            seen &= j > i - window
        q = x[rows].view(T, p.heads, share, p.dim)
        s = torch.einsum("thgd,hnd->hgtn", q, k) * scale
        w = torch.nan_to_num(s.masked_fill(~seen, -float("inf")).softmax(-1))
        reach = (torch.einsum("thgd,hnd->hgtn", q.abs(), k.abs()) * abs(scale)).masked_fill(~seen, 0).amax(-1)
        score = reach * ((p.dim + 8) * 2.0 ** -23 + 2.0 ** -18 * (Q.dtype is torch.bfloat16))
        lost = 2.0 ** -40 * 127 * seen.sum(1) * (w * vs[:, None, None]).amax(-1)
        y = torch.einsum("hgtn,hnd->hgtd", w, v)
        spread = torch.einsum("hgtn,hnd->hgtd", w, v.abs())
        off = spread * (2.0 ** -11 + 2.0 ** -15 + 2 * score[..., None]) + lost[..., None]
        o[rows] = y.permute(2, 0, 1, 3).reshape(T, -1, p.dim)
        limit[rows] += off.permute(2, 0, 1, 3).reshape(T, -1, p.dim)
    return o, limit + torch.clamp(U[Q.dtype] * o.abs(), min=LEAST[Q.dtype])


def check(libgemm, p, Q, counts, lengths, out=None, **kw):
    """The kernel's result for Q, which is within its limit; values past the
    largest of Q's type are infinities."""
    got = p.attend(Q, counts, lengths, out=out, **kw)
    assert libgemm.debug_status() == libgemm.OK
    want, limit = attention(p, Q, counts, lengths, **kw)
    held, most = got.double(), torch.finfo(Q.dtype).max
    inside, past = want.abs() + limit <= most, want.abs() - limit > most * (1 + U[Q.dtype])
    assert torch.isfinite(held[inside]).all() and torch.equal(held[past], torch.copysign(torch.full_like(want, float("inf")), want)[past])
    worst = ((held - want).abs() / limit)[inside].max().item() if inside.any() else 0.0
    assert worst <= 1, worst
    return got
