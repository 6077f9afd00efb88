"""The operators around a 4-bit cache of keys and values, as measured work.

Four operators of a serving step, in the order in which it runs them, each with
its plain form (elementary torch operations in 32 bits, angles in 64) and the
library's own:

  kv_plan        requests' lengths and new tokens to row offsets, positions,
                 slots of the cache and page table entries, whose pages come
                 off a stack of free ones
  rotary         rows of queries and keys turned by their positions (or back,
                 which is the gradient), whole heads or a part, two layouts of
                 the pairs, frequencies scaled for long contexts
  kv4_append     new keys and values quantised to 4 bits into a paged cache,
                 one scale per token and head, and the touched pages read back
  kv4_attention  attention of ragged queries over that cache

Layout of the cache: uint8 [pages][heads][page * (dim + 4)], a page's keys,
values, bfloat16 key scales and value scales of one head one after another.
Code u = c + 8, c in [-7, 7].  Keys: element d of token t is nibble d % 2 of byte
t * dim / 2 + d % 32 / 8 * dim / 8 + d / 32 * 4 + d % 8 / 2.  Values: nibble
d % 2 of byte t / 16 * 8 * dim + t % 16 / 8 * 4 * dim + (4 * (d % 64 / 8) +
t % 8 / 2) * dim / 8 + d / 64 * 8 + d % 8 / 4 * 4 + t % 2 * 2 + d % 4 / 2.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -126


def listed():
    return [
        # a decoding step of 64 requests: latency
        dict(name="plan 64x1", op="kv_plan", batch=64, new=1, past=4000, page=64),
        # a wave of ragged prompts, short pages
        dict(name="plan 1000x512", op="kv_plan", batch=1000, new=512, past=700, page=16),
        # a small model's decoding step: latency
        dict(name="rotate 16x1", op="rotary", batch=16, new=1, past=1000, q_heads=16, kv_heads=4, dim=64, part=64,
             layout="half", base=10000.0, scaling="none", factor=1.0, original=0, inverse=False, type="bf16"),
        # prompts of a long-context model
        dict(name="rotate 4x4096", op="rotary", batch=4, new=4096, past=100000, q_heads=32, kv_heads=8, dim=128, part=128,
             layout="half", base=500000.0, scaling="yarn", factor=8.0, original=8192, inverse=False, type="bf16"),
        # an odd number of rows, a quarter of each head, pairs of neighbours, far positions
        dict(name="rotate 3x777 part", op="rotary", batch=3, new=777, past=1000000, q_heads=12, kv_heads=12, dim=128, part=32,
             layout="interleaved", base=10000.0, scaling="linear", factor=4.0, original=0, inverse=False, type="fp16"),
        # the gradient in a training step
        dict(name="rotate back 8x2048", op="rotary", batch=8, new=2048, past=1, q_heads=16, kv_heads=4, dim=64, part=64,
             layout="half", base=10000.0, scaling="none", factor=1.0, original=0, inverse=True, type="bf16"),
        # a decoding step's write: one token for each of 64 sequences
        dict(name="append4 64x1", op="kv4_append", batch=64, new=1, past=4000, heads=8, dim=128, page=64, type="bf16"),
        # prompts being taken in, ragged
        dict(name="append4 4x4096", op="kv4_append", batch=4, new=4096, past=33, heads=8, dim=128, page=64, type="bf16"),
        # one short sequence's decoding step: latency
        dict(name="attend4 1x1 over 1000", op="kv4_attention", batch=1, new=1, length=1000, q_heads=8, kv_heads=2,
             dim=128, page=16, type="bf16", causal=True, window=0),
        # a full batch of ragged sequences decoding
        dict(name="attend4 64x1 over 8192", op="kv4_attention", batch=64, new=1, length=8192, q_heads=64, kv_heads=8,
             dim=128, page=64, type="bf16", causal=True, window=0),
        # one long sequence decoding, small heads
        dict(name="attend4 1x1 over 200001", op="kv4_attention", batch=1, new=1, length=200001, q_heads=16, kv_heads=4,
             dim=64, page=32, type="fp16", causal=True, window=0),
        # a chunk of long prompts
        dict(name="attend4 4x1000 over 8192", op="kv4_attention", batch=4, new=1000, length=8192, q_heads=32, kv_heads=8,
             dim=128, page=64, type="bf16", causal=True, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["kv_plan", "rotary", "rotary", "kv4_append", "kv4_append", "kv4_attention", "kv4_attention", "kv4_attention"])
    page = rng.choice([16, 32, 64, 128])
    if op == "kv_plan":
        new = _log(rng, 1, 4096)
        return dict(op=op, batch=_log(rng, 1, max(1, min(2000, 500000 // new))), new=new, past=_log(rng, 1, 8192), page=page)
    kind = rng.choice(["bf16", "fp16"])
    if op == "rotary":
        heads = rng.choice([1, 2, 4, 8])
        q_heads, dim, new = heads * rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 80, 96, 128, 256]), _log(rng, 1, 4096)
        most = max(1, 9216 * 40 * 128 // (new * (q_heads + heads) * dim * (2 if kind == "fp32" else 1)))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, batch=_log(rng, 1, min(128, most)), new=new, past=_log(rng, 1, 1000000), q_heads=q_heads,
                    kv_heads=heads, dim=dim, part=rng.choice([dim, dim, dim // 2, dim // 4]), layout=rng.choice(["half", "interleaved"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 10.0]),
                    original=rng.choice([2048, 4096, 8192]) if scaling == "yarn" else 0, inverse=rng.random() < 0.3,
                    type=rng.choice([kind, kind, "fp32"]))
    dim = rng.choice([64, 128])
    if op == "kv4_append":
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


def _pages(tokens, page):
    return -(-tokens // page)


def _past(case):
    return [max(0, p - 1 - 11 * b % 29) for b, p in enumerate(_ragged(case["past"], case["batch"]))]


def _plan_counts(case):
    """New tokens (every ninth request rests), and those in the cache."""
    return [0 if b % 9 == 5 else n for b, n in enumerate(_ragged(case["new"], case["batch"]))], _past(case)


def _append_counts(case):
    new, past = _ragged(case["new"], case["batch"]), _past(case)
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
    if case["op"] == "kv_plan":
        new, past = _plan_counts(case)
        taken = sum(_pages(p + t, case["page"]) - _pages(p, case["page"]) for p, t in zip(past, new))
        # lengths and counts in, offsets, firsts and lengths out; positions and slots; pages off the stack into the
        # table, and the entry of the page that a request was in
        return {"bytes": 20 * case["batch"] + 12 * sum(new) + 8 * taken + 4 * case["batch"], "flops": 2 * sum(new)}
    es = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    if case["op"] == "rotary":
        rows, heads = sum(_ragged(case["new"], case["batch"])), case["q_heads"] + case["kv_heads"]
        return {"bytes": rows * (2 * es * heads * case["dim"] + 4), "flops": 3 * rows * heads * case["part"]}
    if case["op"] == "kv4_append":
        new, past, back = _append_counts(case)
        row, held = 2 * case["heads"] * case["dim"], case["heads"] * (case["dim"] + 4)
        read = sum(p + t - b for p, t, b in zip(past, new, back))
        return {"bytes": sum(new) * (es * row + held) + read * (held + es * row), "flops": 4 * row * sum(new)}
    new, lengths = _attention_counts(case)
    pairs, tokens = _pairs(case)
    return {"bytes": tokens * case["kv_heads"] * (case["dim"] + 4) + 2 * es * sum(new) * case["q_heads"] * case["dim"],
            "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# ---- inputs ------------------------------------------------------------------

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _shuffled(pages, g):
    return torch.randperm(pages, generator=g, device="cuda").to(torch.int32)


def _table(batch, width, g):
    """A page table over a shuffled pool with a few pages to spare."""
    pages = batch * width + 3
    return _shuffled(pages, g)[: batch * width].view(batch, width).contiguous(), pages


def _cache(pages, heads, case, g):
    """A cache in use: codes of about normal values, scales of tokens that differ.
    (Every element's code is drawn alike, so no order of them matters here.)"""
    page, dim = case["page"], case["dim"]
    data = torch.empty((pages, heads, page * (dim + 4)), dtype=torch.uint8, device="cuda")
    for part in data.view(-1, page * (dim + 4)).split(1 << 16):
        u = torch.randn(part.shape[0], page * dim, 2, generator=g, device="cuda").mul_(2.6).round_().clamp_(-7, 7).add_(8.0)
        part[:, : page * dim] = (u[..., 0] + 16.0 * u[..., 1]).to(torch.uint8)
        s = torch.randn(part.shape[0], 2 * page, generator=g, device="cuda").mul_(0.4).exp_().mul_(0.3).to(torch.bfloat16)
        part[:, page * dim:] = s.view(torch.uint8)
    return data


def _handle(s):
    from accelerator_gb300 import lowbit
    return lowbit.Kv4Cache(s["data"], s["page"], s["dim"])


def _frequencies(case):
    """Radians a position of each pair, and the factor of the result, in 64 bits."""
    part, base, factor = case["part"], case["base"], case["factor"]
    at = torch.arange(0, part, 2, dtype=torch.float64, device="cuda") / part
    if case["scaling"] == "ntk" and part > 2:
        base = base * factor ** (part / (part - 2))
    f = base ** -at
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "yarn":
        turns = case["original"] * f / (2 * math.pi)
        kept = ((turns - 1.0) / 31.0).clamp(0, 1)
        f = f / factor * (1 - kept) + f * kept
    return f, 0.1 * math.log(factor) + 1.0 if case["scaling"] == "yarn" else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def normal(*shape, spread=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * spread)

    if case["op"] == "kv_plan":
        new, past = _plan_counts(case)
        held = [_pages(p, case["page"]) for p in past]
        width = max(_pages(p + t, case["page"]) for p, t in zip(past, new)) + 1
        taken = sum(_pages(p + t, case["page"]) for p, t in zip(past, new)) - sum(held)
        pages = _shuffled(sum(held) + taken + 5, g)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda") < _ints(held)[:, None]] = pages[: sum(held)]
        s.update(table=table, lengths=_ints(past), counts=_ints(new), free=pages[sum(held):].contiguous(),
                 available=_ints([taken + 5]), tokens=sum(new))
        return s
    dt = TYPES[case["type"]]
    if case["op"] == "rotary":
        new, past = _ragged(case["new"], case["batch"]), _past(case)
        starts = _ints(_offsets(new))
        row = torch.arange(sum(new), device="cuda")
        seq = torch.searchsorted(starts[1:].long(), row, right=True)
        s["positions"] = (row - starts.long()[seq] + _ints(past).long()[seq]).to(torch.int32)
        # queries and keys as they leave a joint projection: two slices of one array
        both = normal(sum(new), case["q_heads"] + 2 * case["kv_heads"], case["dim"]).to(dt)
        s["Q"], s["K"] = both[:, : case["q_heads"]], both[:, case["q_heads"]: case["q_heads"] + case["kv_heads"]]
        s["frequencies"], s["magnitude"] = _frequencies(case)
        if own:
            from accelerator_gb300 import sequences
            s["handle"] = sequences.Rotary(case["part"], base=case["base"], layout=case["layout"],
                                           scaling=None if case["scaling"] == "none" else case["scaling"],
                                           factor=case["factor"], original=case["original"])
    elif case["op"] == "kv4_append":
        new, past, back = _append_counts(case)
        width = max(_pages(p + t, case["page"]) for p, t in zip(past, new))
        s["table"], pages = _table(case["batch"], width, g)
        s["data"] = _cache(pages, case["heads"], case, g)
        s.update(starts=_ints(_offsets(new)), first=_ints(past), most=max(new),
                 back_starts=_ints(_offsets([p + t - b for p, t, b in zip(past, new, back)])), back_first=_ints(back),
                 back_tokens=sum(p + t - b for p, t, b in zip(past, new, back)))
        # keys and values as they leave a joint projection: two slices of one array
        both = normal(sum(new), 2, case["heads"], case["dim"]).to(dt)
        s["K"], s["V"] = both[:, 0], both[:, 1]
        if own:
            s["handle"] = _handle(s)
    else:
        new, lengths = _attention_counts(case)
        width = max(_pages(n, case["page"]) for n in lengths)
        s["table"], pages = _table(case["batch"], width, g)
        s["data"] = _cache(pages, case["kv_heads"], case, g)
        s.update(starts=_ints(_offsets(new)), lengths=_ints(lengths), most=max(new), longest=max(lengths))
        s["Q"] = normal(sum(new), case["q_heads"], case["dim"], spread=1.5).to(dt)
        if own:
            s["handle"] = _handle(s)
    return s


# ---- the plain forms -----------------------------------------------------------

def _plain_plan(s):
    page, table, lengths, counts = s["page"], s["table"], s["lengths"].long(), s["counts"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    starts = torch.cat([zero, counts.cumsum(0)])
    after = lengths + counts
    held, need = (lengths + page - 1) // page, (after + page - 1) // page
    taken = (need - held).cumsum(0)
    column = torch.arange(table.shape[1], device=table.device)
    fresh = (column >= held[:, None]) & (column < need[:, None])
    at = s["available"].long() - 1 - (taken - need + held)[:, None] - (column - held[:, None])
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].shape[0] - 1)], table))
    row = torch.arange(s["tokens"], device=table.device)
    seq = torch.searchsorted(starts[1:], row, right=True)
    position = row - starts[seq] + lengths[seq]
    slot = table[seq, position // page].long() * page + position % page
    return {"starts": starts.to(torch.int32), "first": s["lengths"].clone(), "lengths": after.to(torch.int32),
            "positions": position.to(torch.int32), "slots": slot, "available": s["available"] - taken[-1:].to(torch.int32),
            "table": table}


def _plain_rotary(s):
    part, half = s["part"], s["part"] // 2
    angle = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = (angle.cos() * s["magnitude"]).float()[:, None], (angle.sin() * s["magnitude"]).float()[:, None]
    if s["inverse"]:
        sin = -sin

    def turned(x):
        y = x.float()
        if s["layout"] == "half":
            a, b = y[..., :half], y[..., half:part]
            return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., part:]], -1).to(x.dtype)
        a, b = y[..., 0:part:2], y[..., 1:part:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., part:]], -1).to(x.dtype)

    return {"q": turned(s["Q"]), "k": turned(s["K"])}


def _unpacked(data, page, dim):
    """Codes c of keys and values as float32 [..., page, dim], and their scales [..., page]."""
    lead, half = data.shape[:-1], page * dim // 2

    def nibbles(x):
        return torch.stack([x & 15, x >> 4], -1).float() - 8.0

    k = nibbles(data[..., :half].reshape(-1, page, 4, dim // 32, 4))                     # t, chunk, word, byte, nibble
    k = k.transpose(2, 3).reshape(*lead, page, dim)
    v = nibbles(data[..., half: 2 * half].reshape(-1, page // 16, 2, 8, 4, dim // 64, 2, 2, 2))
    v = v.permute(0, 1, 2, 4, 7, 5, 3, 6, 8, 9).reshape(*lead, page, dim)                # block, half, pair, odd; 64s, chunk, word, byte, nibble
    scales = data[..., 2 * half:].contiguous().view(torch.bfloat16).float()
    return k, v, scales[..., :page], scales[..., page:]


def _packed(k, v, ks, vs, page, dim):
    """The inverse of _unpacked."""
    lead = k.shape[:-2]

    def bytes_of(c):
        u = (c + 8.0).to(torch.uint8)
        return u[..., 0] | u[..., 1] << 4

    k = bytes_of(k.reshape(-1, page, dim // 32, 4, 4, 2)).transpose(2, 3).reshape(*lead, -1)
    v = bytes_of(v.reshape(-1, page // 16, 2, 4, 2, dim // 64, 8, 2, 2, 2))
    v = v.permute(0, 1, 2, 6, 3, 5, 7, 4, 8).reshape(*lead, -1)
    return torch.cat([k, v, torch.cat([ks, vs], -1).to(torch.bfloat16).view(torch.uint8)], -1)


def _quantised(x):
    """Codes and scales of rows (the last dimension)."""
    scale = (x.abs().amax(-1, keepdim=True) / 7.0).to(torch.bfloat16).float()
    c = torch.where(scale < TINY, 0.0, (x / scale).round().clamp(-7, 7))
    return c, torch.where(scale < TINY, 0.0, scale)[..., 0]


def _plain_append(s):
    page, dim, data = s["page"], s["dim"], s["data"]
    table, first = s["table"].long(), s["first"].long()
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    blocks = torch.arange((s["most"] + page - 2) // page + 1, device=data.device)
    block = torch.minimum(first[:, None] // page + blocks, ((first + count - 1) // page)[:, None])   # sequence, touched page
    at = table.gather(1, block)
    pos = block[:, :, None] * page + torch.arange(page, device=data.device)
    fresh = ((pos >= first[:, None, None]) & (pos < (first + count)[:, None, None]))[:, :, None]     # sequence, page, head, token
    row = (s["starts"][:-1].long()[:, None, None] + pos - first[:, None, None]).clamp(0, s["K"].shape[0] - 1)
    k, v, ks, vs = _unpacked(data[at], page, dim)
    put = []
    for x, codes, scales in ((s["K"], k, ks), (s["V"], v, vs)):
        c, scale = _quantised(x.float())
        put += [torch.where(fresh[..., None], c[row].transpose(2, 3), codes), torch.where(fresh, scale[row].transpose(2, 3), scales)]
    data[at] = _packed(put[0], put[2], put[1], put[3], page, dim)
    row = torch.arange(s["back_tokens"], device=data.device)
    seq = torch.searchsorted(s["back_starts"][1:].long(), row, right=True)
    pos = row - s["back_starts"].long()[seq] + s["back_first"].long()[seq]
    # the touched pages once more, as they are now, and from them the rows that are read back
    k, v, ks, vs = _unpacked(data[at], page, dim)
    where = (seq, pos // page - first[seq] // page, slice(None), pos % page)
    return {n: (c[where] * scale[where][..., None]).to(s["K"].dtype) for n, c, scale in (("k", k, ks), ("v", v, vs))}


def _plain_attention(s):
    q, heads, dim, page = s["Q"], s["kv_heads"], s["dim"], s["page"]
    table, lengths, starts = s["table"].long(), s["lengths"].long(), s["starts"].long()
    batch, longest, most = table.shape[0], s["longest"], s["most"]
    k, v, ks, vs = _unpacked(s["data"][table[:, : -(-longest // page)]], page, dim)

    def dense(codes, scales):       # sequence, head, token, dim
        return codes.mul_(scales[..., None]).transpose(1, 2).reshape(batch, heads, -1, dim)[:, :, :longest]

    count = starts[1:] - starts[:-1]
    step = torch.arange(most, device=q.device)
    row = (starts[:-1, None] + step).clamp(max=q.shape[0] - 1)
    x = q[row].float().view(batch, most, heads, -1, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, -1, dim)
    score = torch.matmul(x, dense(k, ks).transpose(2, 3)).mul_(1.0 / math.sqrt(dim))
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
    o = torch.matmul(p.view(batch, heads, -1, longest), dense(v, vs)).view(batch, heads, -1, most, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, most, -1, dim)
    every = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(starts[1:], every, right=True)
    return o[seq, every - starts[seq]].to(q.dtype)


def run(state):
    s = state
    if own:
        from accelerator_gb300 import lowbit, sequences
        if s["op"] == "kv_plan":
            p = sequences.kv_plan(s["table"], s["lengths"], s["counts"], s["free"], s["available"], s["page"], s["tokens"])
            return {"starts": p.starts, "first": p.first, "lengths": p.lengths, "positions": p.positions, "slots": p.slots,
                    "available": p.available, "table": s["table"]}
        if s["op"] == "rotary":
            q, k = sequences.rotary(s["Q"], s["K"], s["positions"], s["handle"], inverse=s["inverse"])
            return {"q": q, "k": k}
        if s["op"] == "kv4_append":
            lowbit.kv_append(s["handle"], s["K"], s["V"], s["table"], s["starts"], s["first"])
            k, v = lowbit.kv_read(s["handle"], s["table"], s["back_starts"], s["back_first"], s["back_tokens"],
                                  dtype=s["K"].dtype)
            return {"k": k, "v": v}
        return lowbit.kv_attention(s["Q"], s["handle"], s["table"], s["starts"], s["lengths"], causal=s["causal"],
                                   window=s["window"])
    return {"kv_plan": _plain_plan, "rotary": _plain_rotary, "kv4_append": _plain_append,
            "kv4_attention": _plain_attention}[s["op"]](s)


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_rotary(s):
    """Each pair as a complex number times magnitude * exp(i * position * frequency)."""
    part, out = s["part"], {}
    i = torch.arange(part // 2, dtype=torch.float64, device="cuda")
    base, factor = s["base"], s["factor"]
    if s["scaling"] == "ntk" and part > 2:
        base = base * factor ** (part / (part - 2))
    f = torch.exp(-2.0 * i / part * math.log(base))
    length = 2 * math.pi / f                                   # of a turn, in positions
    if s["scaling"] == "linear":
        f = f / factor
    size = 1.0
    if s["scaling"] == "yarn":                                 # from 32 turns in the original context on as it was, under 1 stretched
        ramp = torch.clamp((s["original"] / length - 1) / (32 - 1), 0, 1)
        f = f * (ramp + (1 - ramp) / factor)
        size = 1 + 0.1 * math.log(factor)
    a = s["positions"].double()[:, None, None] * (-f if s["inverse"] else f)
    by = torch.polar(torch.full_like(a, size), a)
    for name, x in (("q", s["Q"].double()), ("k", s["K"].double())):
        y = x.clone()
        if s["layout"] == "half":
            z = torch.complex(x[..., : part // 2], x[..., part // 2: part]) * by
            y[..., : part // 2], y[..., part // 2: part] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., :part].reshape(*x.shape[:2], -1, 2).contiguous()) * by
            y[..., :part] = torch.view_as_real(z).flatten(-2)
        out[name] = y
    return out


def _elements(s, pages, h, tokens):
    """(keys, values) of the first `tokens` tokens of a list of pages, head h, in
    64 bits, byte by byte as the module's text gives the layout."""
    page, dim = s["page"], s["dim"]
    t, d = torch.arange(page, device="cuda")[:, None], torch.arange(dim, device="cuda")
    places = (t * (dim // 2) + d % 32 // 8 * (dim // 8) + d // 32 * 4 + d % 8 // 2,
              page * dim // 2 + t // 16 * 8 * dim + t % 16 // 8 * 4 * dim + (4 * (d % 64 // 8) + t % 8 // 2) * (dim // 8)
              + d // 64 * 8 + d % 8 // 4 * 4 + t % 2 * 2 + d % 4 // 2)
    record, found = s["data"][pages, h], []
    for n, at in enumerate(places):
        u = record[:, at.flatten()].view(-1, page, dim).long() >> (4 * (d % 2)) & 15
        scale = record[:, page * (dim + 2 * n): page * (dim + 2 * n + 2)].contiguous().view(torch.bfloat16).double()
        found.append(((u - 8).double() * scale[..., None]).view(-1, dim)[:tokens])
    return found


def _exact_append(s):
    new, past, back = _append_counts(s)
    outs, at = {"k": [], "v": []}, 0
    for b in range(s["batch"]):
        lo, page = back[b], s["page"]
        pages = s["table"][b, lo // page: _pages(past[b] + new[b], page)].long()
        for n, (name, x) in enumerate((("k", s["K"]), ("v", s["V"]))):
            old = torch.stack([_elements(s, pages[:1], h, past[b] - lo)[n] for h in range(s["heads"])], 1)
            x = x[at: at + new[b]].double()
            scale = (x.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).double()
            c = torch.clamp(torch.round(x / torch.where(scale < TINY, 1.0, scale)), -7, 7)
            outs[name] += [old, torch.where(scale < TINY, 0.0, c * scale)]
        at += new[b]
    return {name: torch.cat(rows) for name, rows in outs.items()}


def _exact_attention(s):
    new, lengths = _attention_counts(s)
    group, at, out = s["q_heads"] // s["kv_heads"], 0, []
    for b in range(s["batch"]):
        n, t = lengths[b], new[b]
        pages = s["table"][b, : _pages(n, s["page"])].long()
        o = torch.zeros((t, s["q_heads"], s["dim"]), dtype=torch.float64, device="cuda")
        i = torch.arange(t, device="cuda")[:, None] + (n - t)
        j = torch.arange(n, device="cuda")
        hide = torch.zeros((t, n), dtype=torch.bool, device="cuda")
        if s["causal"]:
            hide |= j > i
        if s["window"]:
            hide |= j <= i - s["window"]
        for h in range(s["kv_heads"]):
            k, v = _elements(s, pages, h, n)
            for r in range(h * group, (h + 1) * group):
                a = (s["Q"][at: at + t, r].double() @ k.t()) / math.sqrt(s["dim"])
                o[:, r] = torch.softmax(a.masked_fill(hide, -math.inf), -1) @ v
        out.append(o)
        at += t
    return torch.cat(out)


def exact(case, seed):
    if case["op"] == "kv_plan":        # whole numbers, which are compared as they are
        return None
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "kv4_append": _exact_append, "kv4_attention": _exact_attention}[case["op"]](s)
