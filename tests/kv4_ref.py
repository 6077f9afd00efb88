"""The paged 4-bit cache: its layout element by element, the rule of its codes,
and attention over it in 64 bits with a limit on each row's error."""
import numpy as np
import torch

from kv_ref import LEAST, U, ints, offsets

TINY = 2.0 ** -126


def places(page, dim):
    """(byte, nibble) in a record of each token's elements, of keys and of values."""
    t, d = np.arange(page)[:, None], np.arange(dim)[None]
    keys = t * dim // 2 + d % 32 // 8 * (dim // 8) + d // 32 * 4 + d % 8 // 2
    values = page * dim // 2 + t // 16 * (8 * dim) + t % 16 // 8 * (4 * dim) + (4 * (d % 64 // 8) + t % 8 // 2) * (dim // 8) \
        + d // 64 * 8 + d % 8 // 4 * 4 + t % 2 * 2 + d % 4 // 2
    return [torch.from_numpy(x.astype(np.int64)) for x in (keys, values)], torch.from_numpy(d % 2).expand(page, dim)


def pack(codes, scales, page, dim):
    """Records of codes c ([pages, heads, page, dim], int64) and bfloat16 scales, of keys and of values."""
    pages, heads = codes[0].shape[:2]
    data = torch.zeros((pages, heads, page * (dim + 4)), dtype=torch.int64)
    at, nibble = places(page, dim)
    for c, byte in zip(codes, at):
        u = (c.cpu() + 8) << (4 * nibble)
        data.scatter_add_(2, byte.flatten().expand(pages, heads, -1), u.reshape(pages, heads, -1))
    data = data.to(torch.uint8)
    data[:, :, page * dim:] = torch.cat([s.cpu() for s in scales], 2).contiguous().view(torch.uint8)
    return data


def unpack(data, page, dim):
    """The inverse: ([keys, values] codes as int64, [keys, values] scales as bfloat16)."""
    data = data.cpu()
    at, nibble = places(page, dim)
    codes = [(data[:, :, byte.flatten()].long().view(*data.shape[:2], page, dim) >> (4 * nibble) & 15) - 8 for byte in at]
    scales = data[:, :, page * dim:].contiguous().view(torch.bfloat16)
    return codes, [scales[:, :, :page], scales[:, :, page:]]


def quantise(x):
    """Codes and bfloat16 scales of rows x (any type, CPU): the rule of the header."""
    x = x.float()
    top = x.abs().amax(-1)
    top = torch.where(torch.isnan(x).any(-1), float("nan"), top)
    s = (top * torch.tensor(1.0 / 7.0, dtype=torch.float32)).to(torch.bfloat16)
    bad, small = ~torch.isfinite(top), s.float() < TINY
    c = torch.clamp(torch.round(x / s.float()[..., None]), -7, 7)
    c = torch.where((bad | small)[..., None], 0.0, c).long()
    return c, torch.where(bad, float("nan"), torch.where(small, 0.0, s.float())).to(torch.bfloat16)


class Paged4:
    """A 4-bit cache of random codes and scales of about 0.3 (`codes`, `scales`
    may be written over; `load` brings them to the GPU) and a page table in a
    shuffled order."""

    def __init__(self, batch, width, heads, dim, page, seed=0, spare=3):
        from accelerator_gb300 import lowbit
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        pages, self.page, self.heads, self.dim = batch * width + spare, page, heads, dim
        shape = (pages, heads, page, dim)
        self.codes = [self.normal(*shape).mul_(2.6).round_().clamp_(-7, 7).long() for _ in range(2)]
        self.scales = [self.normal(*shape[:3]).mul_(0.5).exp_().mul_(0.3).to(torch.bfloat16) for _ in range(2)]
        self.table = torch.randperm(pages, generator=self.g, device="cuda")[:batch * width].view(batch, width).to(torch.int32)
        self.cache = lowbit.Kv4Cache.empty(pages, heads, dim, page)
        self.load()

    def load(self):
        self.cache.data.copy_(pack(self.codes, self.scales, self.page, self.dim))

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
    """(o, limit) of the rows of Q over the Paged4 p, in 64 bits.  The limit on
    |got - o| of a row, over the n tokens j that it sees with normalised weights
    w_j, codes c, u = c + 8 under 16, scales s_j:
      scores     q.u - 8 q is summed in binary32: dim + 8 roundings of 2^-23 of the
                 sum of magnitudes, |q| (16 + |c|) s at most; a bfloat16 query's
                 elements under 2^-14 of the row's largest lose 2^-25 of that
                 largest each; a score's error moves its weight, and their sum
      weights    w_j s_j is rounded to binary16 (of many rows w_j times the largest
                 s of its 16 tokens): by 2^-11 of itself, or by 2^-25 where 2^12 is
                 the largest product of a weight and a scale of the same 16 tokens,
                 times |c| <= 8
      sums       p u and 8 p apart, in binary32: a chain of n / 64 products of 16 tokens
                 or fewer (four warps share them, or one step takes 128), and 64 steps to
                 join; each loses at most 2^-22 of the sum of magnitudes, 24 s_j w_j
      the rest   exp2 and the sum of the weights: under 2^-15
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

        def dense(which):                                             # head, token, dim; head, token
            c = p.codes[which].to("cuda")[pages].double().transpose(0, 1).reshape(p.heads, -1, p.dim)[:, :n]
            s = p.scales[which].to("cuda")[pages].double().transpose(0, 1).reshape(p.heads, -1)[:, :n]
            return c, s

        (kc, ks), (vc, vs) = dense(0), dense(1)
        k, v = kc * ks[..., None], vc * vs[..., None]
        i = torch.arange(T, device="cuda")[:, None] + (n - T)
        j = torch.arange(n, device="cuda")[None]
        seen = (i >= 0) & ((j <= i) if causal else (j >= 0))
        if window:
            seen &= j > i - window
        q = x[rows].view(T, p.heads, share, p.dim)
        s = torch.einsum("thgd,hnd->hgtn", q, k) * scale
        w = torch.nan_to_num(s.masked_fill(~seen, -float("inf")).softmax(-1))
        reach = torch.einsum("thgd,hnd->hgtn", q.abs(), (16 + kc.abs()) * ks[..., None]) * abs(scale)
        reach = reach.masked_fill(~seen, 0).amax(-1)
        score = reach * ((p.dim + 8) * 2.0 ** -23 + 2.0 ** -18 * (Q.dtype is torch.bfloat16))
        pad = -n % 16
        w16, s16 = (torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (-1, 16)).amax(-1) for x in (w, vs))
        lost = 2.0 ** -37 * 8 * seen.sum(1) * (w16 * s16[:, None, None]).amax(-1)
        chain = (n / 64 + 64) * 2.0 ** -22 * 24 * (w * vs[:, None, None]).sum(-1)
        y = torch.einsum("hgtn,hnd->hgtd", w, v)
        spread = torch.einsum("hgtn,hnd->hgtd", w, v.abs())
        off = spread * (2.0 ** -11 + 2.0 ** -15 + 2 * score[..., None]) + (lost + chain)[..., None]
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
