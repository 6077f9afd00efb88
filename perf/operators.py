"""The operators on operands held in few bits, as measured work.

Four operators of a decoding step, each with its plain form (elementary torch
operations in 32 bits) and the library's own:

  w4_quantize    B (K x N) to 4-bit codes with one bfloat16 scale per `group`
                 rows and column, and back to the values the codes stand for
  gemm_w4        C = X * W for a few rows X and a 4-bit W
  kv_append      new keys and values quantised to 8 bits into a paged cache,
                 one scale per page and head (it grows with the largest
                 magnitude), and the touched pages read back
  kv_attention   attention of ragged queries over that cache

Layouts.  4-bit codes: u = q + 8 for q in [-7, 7], in blocks of 16 columns x
64 rows of 512 bytes, block (n / 16, k / 64); inside a block the 32-bit word
4 * (4 * (n % 8) + k % 32 / 8) + 2 * (k % 64 / 32) + k % 8 / 4 holds the
element in its nibble 4 * (k % 2) + 2 * (k % 4 / 2) + n % 16 / 8.  Scales:
[n / 16][k / group][n % 8][n % 16 / 8].  Cache codes: c + 128 for c in [-127, 127], [page][head][token]
[dim], scales [page][head]; a page table row per sequence.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -126


def listed():
    return [
        # a small projection's weights, float32 checkpoints, an odd width
        dict(name="quantize 1000x1111 g32", op="w4_quantize", k=1000, n=1111, group=32, type="fp32"),
        # loading a large layer's weights
        dict(name="quantize 8192x8192 g128", op="w4_quantize", k=8192, n=8192, group=128, type="bf16"),
        # one token through a small projection: latency
        dict(name="w4 1x1024x1024", op="gemm_w4", m=1, k=1024, n=1024, group=64, type="bf16", out="bf16"),
        # one token through a large layer: the weights' bytes
        dict(name="w4 1x8192x8192", op="gemm_w4", m=1, k=8192, n=8192, group=128, type="bf16", out="bf16"),
        # a few sequences, ragged sizes, fine groups, float32 results
        dict(name="w4 5x4100x5001 g32", op="gemm_w4", m=5, k=4100, n=5001, group=32, type="fp16", out="fp32"),
        # a batch of decoding sequences through the largest layer
        dict(name="w4 16x16384x16384", op="gemm_w4", m=16, k=16384, n=16384, group=128, type="bf16", out="bf16"),
        # a decoding step's write: one token for each of 64 sequences
        dict(name="append 64x1", op="kv_append", batch=64, new=1, past=4000, heads=8, dim=128, page=64, type="bf16"),
        # prompts being taken in, ragged
        dict(name="append 4x4096", op="kv_append", batch=4, new=4096, past=33, heads=8, dim=128, page=64, type="bf16"),
        # one short sequence's decoding step: latency
        dict(name="attend 1x1 over 1000", op="kv_attention", batch=1, new=1, length=1000, q_heads=8, kv_heads=2,
             dim=128, page=16, type="bf16", causal=True, window=0),
        # a full batch of ragged sequences decoding
        dict(name="attend 64x1 over 8192", op="kv_attention", batch=64, new=1, length=8192, q_heads=64, kv_heads=8,
             dim=128, page=64, type="bf16", causal=True, window=0),
        # one long sequence decoding, small heads
        dict(name="attend 1x1 over 200001", op="kv_attention", batch=1, new=1, length=200001, q_heads=16, kv_heads=4,
             dim=64, page=32, type="fp16", causal=True, window=0),
        # a chunk of long prompts
        dict(name="attend 4x1000 over 8192", op="kv_attention", batch=4, new=1000, length=8192, q_heads=32, kv_heads=8,
             dim=128, page=64, type="bf16", causal=True, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["w4_quantize", "gemm_w4", "gemm_w4", "kv_append", "kv_attention", "kv_attention", "kv_attention"])
    if op == "w4_quantize":
        k, n = _log(rng, 200, 8192), _log(rng, 200, 8192)
        return dict(op=op, k=k + (k == 3072), n=n + (n == 3072), group=rng.choice([32, 64, 128]),
                    type=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "gemm_w4":
        k, n = _log(rng, 500, 16384), _log(rng, 500, 16384)
        return dict(op=op, m=_log(rng, 1, 16), k=k + (k == 3072), n=n + (n == 3072), group=rng.choice([32, 64, 128]),
                    type=rng.choice(["bf16", "fp16"]), out=rng.choice(["same", "fp32"]))
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128])
    kind = rng.choice(["bf16", "fp16"])
    if op == "kv_append":
        new = _log(rng, 1, 4096)
        return dict(op=op, batch=_log(rng, 1, max(1, min(128, 16384 // new))), new=new, past=_log(rng, 1, 8192),
                    heads=rng.choice([1, 2, 4, 8]), dim=dim, page=page, type=kind)
    heads = rng.choice([1, 2, 4, 8])
    share = rng.choice([1, 2, 3, 4, 6, 8])
    window = rng.choice([0, 0, 0, 500])
    if rng.random() < 0.6:      # decoding, up to a few tokens at once
        new, batch = rng.choice([1, 1, 1, 2, 5]), _log(rng, 1, 64)
        length = _log(rng, 100, min(200000, 64 * 8192 // batch // new))
    else:                       # prompts
        new, batch = _log(rng, 20, 1000), rng.choice([1, 2, 3, 4])
        share = min(share, 32 // heads)
        length = _log(rng, new, 8192)
    return dict(op=op, batch=batch, new=new, length=max(length, new), q_heads=heads * share, kv_heads=heads, dim=dim,
                page=page, type=kind, causal=new == 1 or rng.random() < 0.75 or window > 0, window=window)


# ---- shapes that follow from a case ----------------------------------------

def _ragged(most, batch):
    """Counts of a batch: `most` for one sequence, down to about an eighth of it for others."""
    return [max(1, most - (b * 37 % batch) * most * 7 // (8 * batch)) for b in range(batch)]


def _offsets(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _append_counts(case):
    new = _ragged(case["new"], case["batch"])
    past = [max(0, p - 1 - 11 * b % 29) for b, p in enumerate(_ragged(case["past"], case["batch"]))]
    back = [p // case["page"] * case["page"] for p in past]          # the touched pages' first tokens
    return new, past, back


def _attention_counts(case):
    lengths = _ragged(case["length"], case["batch"])
    return [min(t, n) for t, n in zip(_ragged(case["new"], case["batch"]), lengths)], lengths


def _pairs(case):
    """(query, key) pairs that the mask leaves, and the cached tokens that any query sees."""
    pairs = tokens = 0
    for t, n in zip(*_attention_counts(case)):
        w = case["window"] or n
        for i in range(t) if case["causal"] else ():
            pairs += min(w, n - t + i + 1)
        pairs += 0 if case["causal"] else t * n
        tokens += min(n, w + t - 1) if case["causal"] else n
    return pairs, tokens


def work(case):
    es = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    if case["op"] == "w4_quantize":
        k, n = case["k"], case["n"]
        held = k * n // 2 + 2 * n * -(-k // case["group"])
        return {"bytes": 2 * es * k * n + 2 * held, "flops": 4 * k * n}
    if case["op"] == "gemm_w4":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": k * n // 2 + 2 * n * -(-k // case["group"]) + es * m * k + m * n * (4 if case["out"] == "fp32" else es),
                "flops": 2 * m * k * n}
    if case["op"] == "kv_append":
        new, past, back = _append_counts(case)
        row = 2 * case["heads"] * case["dim"]
        read = sum(p + t - b for p, t, b in zip(past, new, back))
        return {"bytes": row * (sum(new) * (es + 1) + read * (1 + es)), "flops": 4 * row * sum(new)}
    new, lengths = _attention_counts(case)
    pairs, tokens = _pairs(case)
    return {"bytes": 2 * tokens * case["kv_heads"] * case["dim"] + 2 * es * sum(new) * case["q_heads"] * case["dim"],
            "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# ---- inputs ------------------------------------------------------------------

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(batch, width, g):
    """A page table over a shuffled pool with a few pages to spare."""
    pages = batch * width + 3
    at = torch.randperm(pages, generator=g, device="cuda")[: batch * width]
    return at.to(torch.int32).view(batch, width).contiguous(), pages


def _cache(pages, case, heads, g):
    """A cache in use: codes of about normal values, the scales of pages that differ."""
    shape = (pages, heads, case["page"], case["dim"])
    made = []
    for _ in range(2):
        codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for part in codes.view(-1).split(1 << 28):
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(32.0).round_().clamp_(-127, 127).add_(128.0))
        made.append(codes)
    for spread in (0.5, 0.3):
        made.append(torch.randn(shape[:2], generator=g, device="cuda").mul_(spread).exp_().mul_(0.03))
    return {"k_codes": made[0], "v_codes": made[1], "k_scales": made[2], "v_scales": made[3]}


def _handle(cache):
    from accelerator_gb300 import lowbit
    return lowbit.KvCache(cache["k_codes"], cache["v_codes"], cache["k_scales"], cache["v_scales"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["type"]]
    s = dict(case)

    def normal(*shape, spread=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * spread)

    if case["op"] == "w4_quantize":
        s["B"] = normal(case["k"], case["n"], spread=0.02).to(dt)
    elif case["op"] == "gemm_w4":
        nb, kb = -(-case["n"] // 16), -(-case["k"] // 64)
        words = torch.empty((nb, kb, 32, 4), dtype=torch.int32, device="cuda")
        for part in words.view(-1).split(1 << 24):
            u = normal(part.numel(), 8, spread=2.6).round_().clamp_(-7, 7).add_(8).to(torch.int32)
            part.copy_((u << torch.arange(0, 32, 4, dtype=torch.int32, device="cuda")).sum(1).to(torch.int32))
        scales = (normal(nb, -(-case["k"] // case["group"]), 8, 2, spread=0.25).exp() * 0.008).to(torch.bfloat16)
        x = normal(case["m"], case["k"])
        x[:, 5::97] *= 9.0          # channels of large magnitude, as activations have them
        s.update(X=x.to(dt), words=words, scales=scales)
        if own:
            from accelerator_gb300 import lowbit
            s["W"] = lowbit.W4Matrix(words.view(torch.uint8).view(-1), scales, case["k"], case["n"], case["group"])
    elif case["op"] == "kv_append":
        new, past, back = _append_counts(case)
        width = max(-(-(p + t) // case["page"]) for p, t in zip(past, new))
        s["table"], pages = _table(case["batch"], width, g)
        s["cache"] = _cache(pages, case, case["heads"], g)
        s.update(starts=_ints(_offsets(new)), first=_ints(past), most=max(new),
                 back_starts=_ints(_offsets([p + t - b for p, t, b in zip(past, new, back)])), back_first=_ints(back),
                 back_tokens=sum(p + t - b for p, t, b in zip(past, new, back)))
        # keys and values as they leave a joint projection: two slices of one array
        both = normal(sum(new), 2, case["heads"], case["dim"]).to(dt)
        s["K"], s["V"] = both[:, 0], both[:, 1]
        if own:
            s["handle"] = _handle(s["cache"])
    else:
        new, lengths = _attention_counts(case)
        width = max(-(-n // case["page"]) for n in lengths)
        s["table"], pages = _table(case["batch"], width, g)
        s["cache"] = _cache(pages, case, case["kv_heads"], g)
        s.update(starts=_ints(_offsets(new)), lengths=_ints(lengths), most=max(new), longest=max(lengths))
        s["Q"] = normal(sum(new), case["q_heads"], case["dim"], spread=1.5).to(dt)
        if own:
            s["handle"] = _handle(s["cache"])
    return s


# ---- the plain forms -----------------------------------------------------------

def _plain_quantize(s):
    k, n, group = s["k"], s["n"], s["group"]
    w = s["B"].float()
    w = torch.nn.functional.pad(w, (0, 0, 0, -k % group)).view(-1, group, n)
    scale = (w.abs().amax(1, keepdim=True) / 7.0).to(torch.bfloat16).float()
    q = (w / scale).round().clamp(-7, 7)
    q = torch.where(scale < TINY, torch.zeros_like(q), q)
    return (q * scale).view(-1, n)[:k].to(s["B"].dtype)


def _plain_weights(s):
    """N x K float32 values of the packed codes and scales."""
    k, n, group, words = s["k"], s["n"], s["group"], s["words"]
    nb, kb = words.shape[:2]
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=words.device)
    u = ((words.unsqueeze(-1) >> shifts) & 15).to(torch.uint8)      # block n, block k, lane, word, nibble
    u = u.view(nb, kb, 8, 4, 2, 2, 2, 2, 2).permute(0, 8, 2, 1, 4, 3, 5, 7, 6).reshape(nb * 16, kb * 64)[:n, :k]
    scale = s["scales"].float().permute(0, 3, 2, 1).reshape(nb * 16, -1)[:n]
    scale = scale.repeat_interleave(group, 1)[:, :k]
    return (u.float() - 8.0) * scale


def _plain_gemm_w4(s):
    y = torch.matmul(s["X"].float(), _plain_weights(s).t())
    return y.to(torch.float32 if s["out"] == "fp32" else s["X"].dtype)


def _plain_write(codes, scales, x, s):
    """Quantises the new rows x into the cache's pages, in place."""
    page, table, first = s["page"], s["table"].long(), s["first"].long()
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    blocks = torch.arange((s["most"] + page - 2) // page + 1, device=x.device)
    block = torch.minimum(first[:, None] // page + blocks, ((first + count - 1) // page)[:, None])   # sequence, touched page
    at = table.gather(1, block)
    pos = block[:, :, None] * page + torch.arange(page, device=x.device)
    fresh = (pos >= first[:, None, None]) & (pos < (first + count)[:, None, None])
    row = (s["starts"][:-1].long()[:, None, None] + pos - first[:, None, None]).clamp(0, x.shape[0] - 1)
    new = (x[row].float() * fresh[..., None, None]).transpose(2, 3)              # sequence, page, head, token, dim
    old = codes[at].float() - 128.0
    before = torch.where((block * page < first[:, None])[..., None], scales[at], 0.0)
    scale = torch.maximum(before, new.abs().amax((3, 4)) / 127.0)
    inverse = torch.where(scale < TINY, 0.0, 1.0 / scale)
    put = torch.where(fresh[:, :, None, :, None], (new * inverse[..., None, None]).round().clamp(-127, 127),
                      torch.where((before < scale)[..., None, None], (old * (before * inverse)[..., None, None]).round(), old))
    codes[at] = (put + 128.0).to(torch.uint8)
    scales[at] = scale


def _plain_read(codes, scales, s, dt):
    row = torch.arange(s["back_tokens"], device=codes.device)
    seq = torch.searchsorted(s["back_starts"][1:].long(), row, right=True)
    pos = row - s["back_starts"].long()[seq] + s["back_first"].long()[seq]
    at = s["table"].long()[seq, pos // s["page"]]
    return ((codes[at, :, pos % s["page"]].float() - 128.0) * scales[at][..., None]).to(dt)


def _plain_append(s):
    c, dt = s["cache"], s["K"].dtype
    _plain_write(c["k_codes"], c["k_scales"], s["K"], s)
    _plain_write(c["v_codes"], c["v_scales"], s["V"], s)
    return {"k": _plain_read(c["k_codes"], c["k_scales"], s, dt), "v": _plain_read(c["v_codes"], c["v_scales"], s, dt)}


def _plain_attention(s):
    c, q, heads, dim, page = s["cache"], s["Q"], s["kv_heads"], s["dim"], s["page"]
    table, lengths, starts = s["table"].long(), s["lengths"].long(), s["starts"].long()
    batch, longest, most = table.shape[0], s["longest"], s["most"]
    pages = table[:, : -(-longest // page)]

    def dense(codes, scales):       # sequence, head, token, dim
        x = (codes[pages].float() - 128.0) * scales[pages][..., None, None]
        return x.transpose(1, 2).reshape(batch, heads, -1, dim)[:, :, :longest]

    count = starts[1:] - starts[:-1]
    step = torch.arange(most, device=q.device)
    row = (starts[:-1, None] + step).clamp(max=q.shape[0] - 1)
    x = q[row].float().view(batch, most, heads, -1, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, -1, dim)
    score = torch.matmul(x, dense(c["k_codes"], c["k_scales"]).transpose(2, 3)).mul_(1.0 / math.sqrt(dim))
    score = score.view(batch, heads, -1, most, longest)
    key = torch.arange(longest, device=q.device)
    own_key = (lengths - count)[:, None] + step                      # a query's own position
    seen = (key < lengths[:, None, None]) & (own_key >= 0)[..., None]
    if s["causal"]:
        seen = seen & (key <= own_key[..., None])
    if s["window"]:
        seen = seen & (key > own_key[..., None] - s["window"])
    seen = seen[:, None, None]
    score = score.masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, heads, -1, longest), dense(c["v_codes"], c["v_scales"])).view(batch, heads, -1, most, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, most, -1, dim)
    every = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(starts[1:], every, right=True)
    return o[seq, every - starts[seq]].to(q.dtype)


def run(state):
    s = state
    if own:
        from accelerator_gb300 import lowbit
        if s["op"] == "w4_quantize":
            return lowbit.w4_dequantize(lowbit.w4_quantize(s["B"], s["group"]), dtype=s["B"].dtype)
        if s["op"] == "gemm_w4":
            return lowbit.gemm_w4(s["X"], s["W"], dtype=torch.float32 if s["out"] == "fp32" else s["X"].dtype)
        if s["op"] == "kv_append":
            lowbit.kv_append(s["handle"], s["K"], s["V"], s["table"], s["starts"], s["first"])
            k, v = lowbit.kv_read(s["handle"], s["table"], s["back_starts"], s["back_first"], s["back_tokens"],
                                  dtype=s["K"].dtype)
            return {"k": k, "v": v}
        return lowbit.kv_attention(s["Q"], s["handle"], s["table"], s["starts"], s["lengths"], causal=s["causal"],
                                   window=s["window"])
    return {"w4_quantize": _plain_quantize, "gemm_w4": _plain_gemm_w4, "kv_append": _plain_append,
            "kv_attention": _plain_attention}[s["op"]](s)


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_quantize(s):
    w = s["B"].double()
    out = torch.empty_like(w)
    for k in range(0, s["k"], s["group"]):
        part = w[k: k + s["group"]]
        scale = (part.abs().amax(0) / 7).to(torch.bfloat16).double()
        q = torch.clamp(torch.round(part / scale), -7, 7)
        out[k: k + s["group"]] = torch.where(scale < TINY, 0.0, q * scale)
    return out


def _exact_gemm_w4(s):
    """Sixteen columns at a time, element by element of the layout as the module's text gives it."""
    k = torch.arange(s["k"], device="cuda")
    x, out = s["X"].double(), []
    for block in range(s["words"].shape[0]):
        n = torch.arange(16, device="cuda")[:, None]
        word = s["words"][block].view(-1)[k // 64 * 128 + 4 * (4 * (n % 8) + k % 32 // 8) + 2 * (k % 64 // 32) + k % 8 // 4].long()
        q = (word >> (4 * (4 * (k % 2) + 2 * (k % 4 // 2) + n // 8)) & 15) - 8
        w = q.double() * s["scales"][block][k // s["group"], n % 8, n // 8].double()
        out.append(x @ w.t())
    return torch.cat(out, 1)[:, : s["n"]]


def _exact_append(s):
    new, past, back = _append_counts(s)
    table, page, outs = s["table"].tolist(), s["page"], []
    for codes, scales, x in ((s["cache"]["k_codes"], s["cache"]["k_scales"], s["K"]),
                             (s["cache"]["v_codes"], s["cache"]["v_scales"], s["V"])):
        at, rows = 0, []
        for b in range(s["batch"]):
            end = past[b] + new[b]
            for lo in range(back[b], end, page):
                old = max(0, min(past[b] - lo, page))
                lo_new, hi = lo + old, min(lo + page, end)
                fresh = x[at + lo_new - past[b]: at + hi - past[b]].double()     # token, head, dim
                held = codes[table[b][lo // page], :, :old].double().transpose(0, 1) - 128
                before = scales[table[b][lo // page]].double() * (old > 0)
                scale = torch.maximum(before, fresh.abs().amax((0, 2)) / 127)
                ratio = torch.where(scale > 0, before / scale, 1.0)[None, :, None]
                held = torch.where(ratio < 1, torch.round(held * ratio), held)
                put = torch.round(fresh / torch.where(scale < TINY, 1.0, scale)[None, :, None])
                rows.append(torch.cat([held, put]) * scale[None, :, None])
            at += new[b]
        outs.append(torch.cat(rows))
    return {"k": outs[0], "v": outs[1]}


def _exact_attention(s):
    new, lengths = _attention_counts(s)
    c, group, at, out = s["cache"], s["q_heads"] // s["kv_heads"], 0, []
    for b in range(s["batch"]):
        n, t = lengths[b], new[b]
        pages = s["table"][b, : -(-n // s["page"])].long()
        o = torch.zeros((t, s["q_heads"], s["dim"]), dtype=torch.float64, device="cuda")
        i = torch.arange(t, device="cuda")[:, None] + (n - t)
        j = torch.arange(n, device="cuda")
        hide = torch.zeros((t, n), dtype=torch.bool, device="cuda")
        if s["causal"]:
            hide |= j > i
        if s["window"]:
            hide |= j <= i - s["window"]
        for h in range(s["kv_heads"]):
            k = ((c["k_codes"][pages, h].double() - 128) * c["k_scales"][pages, h].double()[:, None, None]).reshape(-1, s["dim"])[:n]
            v = ((c["v_codes"][pages, h].double() - 128) * c["v_scales"][pages, h].double()[:, None, None]).reshape(-1, s["dim"])[:n]
            for r in range(h * group, (h + 1) * group):
                a = (s["Q"][at: at + t, r].double() @ k.t()) / math.sqrt(s["dim"])
                o[:, r] = torch.softmax(a.masked_fill(hide, -math.inf), -1) @ v
        out.append(o)
        at += t
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"w4_quantize": _exact_quantize, "gemm_w4": _exact_gemm_w4, "kv_append": _exact_append,
            "kv_attention": _exact_attention}[s["op"]](s)
