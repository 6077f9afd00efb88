"""Attention over the paged 4-bit cache against 64 bits: lengths around every
page and tile edge, head layouts, masks that leave rows empty, windows, few rows
and many, whole and joined, strides, scales far apart, NaN where it is seen."""
import pytest
import torch

import kv4_ref as ref
from kv_ref import ints

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, torch.float16, 16), (64, torch.bfloat16, 128), (128, torch.bfloat16, 64), (128, torch.float16, 32)]
layouts = pytest.mark.parametrize("dim,kind,page", LAYOUTS)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_at_every_edge(libgemm, page, dim, kind):
    lengths = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 0, 511]
    p = ref.Paged4(len(lengths), -(-512 // page), 2, dim, page, seed=page + dim)
    for share in (1, 4):
        ref.check(libgemm, p, p.queries(len(lengths), 2 * share, kind), [1] * len(lengths), lengths)


@pytest.mark.parametrize("heads,share", [(1, 1), (1, 16), (1, 17), (2, 8), (3, 5), (5, 3), (8, 1), (1, 40), (2, 9)])
def test_head_layouts(libgemm, heads, share):
    p = ref.Paged4(3, 5, heads, 64, 64, seed=heads + share)
    ref.check(libgemm, p, p.queries(6, heads * share, torch.float16), [1, 2, 3], [200, 77, 300])


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 33), (True, 100), (False, 0)])
@pytest.mark.parametrize("dim,share", [(64, 1), (128, 4), (128, 3)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
def test_prompts(libgemm, dim, share, causal, window, kind):
    counts, lengths = [1, 40, 0, 129, 64, 200, 5], [1, 40, 10, 150, 300, 200, 129]
    p = ref.Paged4(7, 10, 2, dim, 32, seed=dim + share)
    ref.check(libgemm, p, p.queries(sum(counts), 2 * share, kind), counts, lengths, causal=causal, window=window)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing_are_zero(libgemm, causal):
    """More queries than tokens, and empty caches, of few rows and of many."""
    p = ref.Paged4(4, 2, 2, 64, 32, seed=8)
    O = ref.check(libgemm, p, p.queries(49, 6, torch.bfloat16), [5, 3, 40, 1], [2, 0, 30, 0], causal=causal)
    assert (O[:3] == 0).all() and (O[5:18] == 0).all() and (O[-1] == 0).all() and (O[4] != 0).any()
    p = ref.Paged4(3, 2, 1, 128, 64, seed=9)
    O = ref.check(libgemm, p, p.queries(590, 2, torch.float16), [200, 300, 90], [60, 0, 1], causal=causal)
    assert (O[:140] == 0).all() and (O[200:589] == 0).all() and (O[589] != 0).any()


@layouts
@pytest.mark.parametrize("T,share", [(1, 1), (1, 8), (3, 5)])
@pytest.mark.parametrize("window", [0, 9000])
def test_few_rows_of_long_sequences(libgemm, dim, kind, page, T, share, window):
    counts, lengths = [T, T, T, T, 0], [20011, 130, 0, 1, 500]
    p = ref.Paged4(5, -(-20011 // page), 2, dim, page, seed=T + share)
    ref.check(libgemm, p, p.queries(4 * T, 2 * share, kind), counts, lengths, window=window)


@layouts
@pytest.mark.parametrize("counts,lengths", [([300, 0, 41], [3001, 700, 41]), ([1000], [1300]), ([130, 130], [2600, 100])])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 700), (False, 0)])
def test_many_rows_over_few_heads(libgemm, dim, kind, page, counts, lengths, causal, window):
    p = ref.Paged4(len(counts), -(-max(lengths) // page), 1, dim, page, seed=len(counts))
    ref.check(libgemm, p, p.queries(sum(counts), 3, kind), counts, lengths, causal=causal, window=window)


@layouts
def test_many_rows_over_many_blocks(libgemm, dim, kind, page):
    counts, lengths = [300, 513, 700, 90], [4000, 2111, 1900, 90]
    p = ref.Paged4(4, -(-4000 // page), 8, dim, page)
    Q = p.queries(sum(counts), 16, kind)
    ref.check(libgemm, p, Q, counts, lengths)
    ref.check(libgemm, p, Q, counts, lengths, window=333)


@layouts
@pytest.mark.parametrize("rows", [1, 3, 60, 400])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-6, 2.0])
def test_scales_of_any_sign(libgemm, dim, kind, page, rows, scale):
    p = ref.Paged4(1, -(-1500 // page), 2, dim, page)
    ref.check(libgemm, p, p.queries(rows, 4, kind), [rows], [1500], scale=scale)


@layouts
@pytest.mark.parametrize("rows,length", [(4, 300), (60, 300), (500, 1500)])
def test_strided_rows_and_results(libgemm, dim, kind, page, rows, length):
    p = ref.Paged4(1, -(-length // page), 2, dim, page)
    joint = p.queries(rows, 9, kind).flatten(1)
    for shift in (0, 8, 3):
        Q = joint[:, shift:shift + 4 * dim].unflatten(1, (4, dim))
        store = torch.full((rows, 4, dim + 36), float("nan"), dtype=kind, device="cuda")
        ref.check(libgemm, p, Q, [rows], [length], out=store[:, :, shift:shift + dim])
        assert torch.isnan(store[:, :, shift + dim:]).all() and torch.isnan(store[:, :, :shift]).all()
    by_head = torch.empty((4, rows, dim), dtype=kind, device="cuda")
    ref.check(libgemm, p, joint[:, :4 * dim].unflatten(1, (4, dim)), [rows], [length], out=by_head.transpose(0, 1))


@layouts
@pytest.mark.parametrize("rows,length", [(4, 300), (60, 300), (500, 1500), (2, 20000)])
def test_nan_stays_where_it_is_seen(libgemm, dim, kind, page, rows, length):
    """In a query: in its row and head.  In a token's scales: in the rows that see it."""
    p = ref.Paged4(1, -(-length // page), 2, dim, page)
    Q = p.queries(rows, 4, kind)
    want = ref.check(libgemm, p, Q, [rows], [length])
    Q[rows // 2, 3, 5] = float("nan")
    got = p.attend(Q, [rows], [length])
    assert torch.isnan(got[rows // 2, 3]).all()
    got[rows // 2, 3] = want[rows // 2, 3]
    assert torch.equal(got, want)
    Q[rows // 2, 3, 5] = 0.5
    want = p.attend(Q, [rows], [length])
    for which in (0, 1):
        for token in (length - 1, length - rows // 2 - 1, length // 3):
            at = (p.page_of(0, token // page), 1, token % page)
            kept = p.scales[which][at].item()
            p.scales[which][at] = float("nan")
            p.load()
            got = p.attend(Q, [rows], [length])
            hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
            hit[max(0, token - (length - rows)):] = True
            assert torch.isnan(got[hit, 2:]).all()
            assert torch.equal(got[~hit], want[~hit]) and torch.equal(got[:, :2], want[:, :2])
            p.scales[which][at] = kept
    assert libgemm.debug_status() == libgemm.OK


@layouts
@pytest.mark.parametrize("rows", [1, 4, 60, 300])
def test_what_no_row_sees_is_not_used(libgemm, dim, kind, page, rows):
    """NaN, infinities and huge scales in the tokens past the last one, in the pages
    of the pool that are not in the table and in those before every window."""
    length = 700
    p = ref.Paged4(1, -(-length // page) + 1, 2, dim, page)
    Q = p.queries(rows, 8, kind)
    want, inside = (ref.check(libgemm, p, Q, [rows], [length], window=w) for w in (0, 40))
    used = [p.page_of(0, i) for i in range(-(-length // page))]
    for poison in (float("nan"), float("inf"), -float("inf"), 3e38, -3e38):
        for s in p.scales:
            for other in set(range(s.shape[0])) - set(used):
                s[other] = poison
            s[used[-1], :, (length - 1) % page + 1:] = poison
        p.load()
        assert torch.equal(p.attend(Q, [rows], [length]), want)
        first = length - rows - 40 + 1           # the first token that a row sees through its window
        kept = [s.clone() for s in p.scales]
        for s in p.scales:
            for i in range(max(0, first)):
                s[used[i // page], :, i % page] = poison
        p.load()
        assert torch.equal(p.attend(Q, [rows], [length], window=40), inside)
        p.scales = kept
    assert libgemm.debug_status() == libgemm.OK


@layouts
@pytest.mark.parametrize("T,share", [(1, 4), (5, 3), (60, 2)])
@pytest.mark.parametrize("window", [1, 40, 300])
def test_pages_before_the_window_may_be_gone(libgemm, dim, kind, page, T, share, window):
    lengths = [700, 515]
    p = ref.Paged4(2, -(-700 // page), 2, dim, page, seed=window)
    Q = p.queries(2 * T, 2 * share, kind)
    want = ref.check(libgemm, p, Q, [T, T], lengths, window=window)
    for b, n in enumerate(lengths):
        for i in range(max(0, n - T - window + 1) // page):
            p.table[b, i] = -1 if b else p.codes[0].shape[0]
    assert torch.equal(p.attend(Q, [T, T], lengths, window=window), want)
    assert libgemm.debug_status() == libgemm.OK


@layouts
@pytest.mark.parametrize("T,length", [(1, 2000), (4, 900), (60, 700), (300, 900)])
def test_scales_that_differ_by_orders(libgemm, dim, kind, page, T, length):
    """Neighbouring tokens whose scales are 2^20 apart, single ones far above the
    rest, tokens of zeros; scores and weights of any magnitude that float holds."""
    p = ref.Paged4(2, -(-length // page), 1, dim, page, seed=T)
    Q = p.queries(2 * T, 4, kind)
    base = [s.clone() for s in p.scales]

    def with_scales(k, v, **kw):
        for to, by, s in zip(p.scales, (k, v), base):
            to.copy_((s.float() * by).to(torch.bfloat16))
        p.load()
        ref.check(libgemm, p, Q, [T, T], [length, length // 2], **kw)

    one = torch.ones_like(base[0], dtype=torch.float32)
    far = torch.exp2(p.normal(*one.shape).clamp_(-3, 3) * 7)
    with_scales(one, far)
    with_scales(torch.clamp(far, max=2.0), one * 2.0 ** -100)
    with_scales(one, torch.where(p.normal(*one.shape) > 1, 0.0, 1.0))
    with_scales(one * 0, one)
    with_scales(one, one * 0)
    if kind is torch.bfloat16:
        with_scales(one, one * 2.0 ** 100)
        with_scales(one * 2.0 ** 60, one, scale=2.0 ** -62)
        with_scales(one * 2.0 ** -60, far * 2.0 ** 40, scale=2.0 ** 58)


@pytest.mark.parametrize("rows", [5, 60])
@pytest.mark.parametrize("magnitude", [2.0 ** -60, 1.0, 2.0 ** 60])
def test_queries_of_any_magnitude(libgemm, rows, magnitude):
    p = ref.Paged4(1, 20, 2, 128, 16, seed=12)
    Q = p.normal(rows, 4, 128) * magnitude
    Q[:, :, ::7] *= 2.0 ** -20
    ref.check(libgemm, p, Q.to(torch.bfloat16), [rows], [300], scale=float(0.1 / magnitude))


@layouts
@pytest.mark.parametrize("share", [1, 4, 5])
def test_prompts_and_single_tokens_together(libgemm, dim, kind, page, share):
    counts = [1, 1, 700, 1, 0, 1, 1, 33, 1, 1, 1, 2]
    lengths = [900, 17, 700, 1, 300, 0, 513, 40, 1300, 64, 65, 600]
    p = ref.Paged4(len(counts), -(-1300 // page), 2, dim, page, seed=share)
    ref.check(libgemm, p, p.queries(sum(counts), 2 * share, kind), counts, lengths)


@layouts
@pytest.mark.parametrize("rows", [1, 5, 60])
def test_the_same_on_every_run(libgemm, dim, kind, page, rows):
    p = ref.Paged4(2, -(-12000 // page), 2, dim, page)
    Q = p.queries(2 * rows, 4, kind)
    want = p.attend(Q, [rows, rows], [12000, 5000])
    for _ in range(5):
        assert torch.equal(p.attend(Q, [rows, rows], [12000, 5000]), want)


@pytest.mark.parametrize("T,length", [(1, 20000), (60, 3000)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1, 2 ** 64 + 5])
def test_a_window_past_every_token_is_none(libgemm, T, length, window):
    p = ref.Paged4(1, -(-length // 64), 1, 64, 64)
    Q = p.queries(T, 4, torch.float16)
    want = ref.check(libgemm, p, Q, [T], [length])
    assert torch.equal(p.attend(Q, [T], [length], window=window), want)
    assert libgemm.debug_status() == libgemm.OK


@pytest.mark.parametrize("share", [1, 8])
def test_offsets_that_descend_are_reported(libgemm, share):
    from test_kv_offsets import BAD
    from accelerator_gb300 import lowbit
    p = ref.Paged4(5, 20, 1, 64, 16)
    for starts in BAD:
        assert libgemm.debug_status() == libgemm.OK
        lowbit.kv_attention(p.queries(240, share, torch.float16), p.cache, p.table, ints(starts), ints([300] * 5))
        assert libgemm.debug_status() == libgemm.ERR_INDEX


@layouts
def test_many_sequences_in_one_line(libgemm, dim, kind, page):
    """More sequences than a block has threads, of none to three rows, of every
    length around a step's and a page's end, some empty."""
    n = 400
    lengths = [(b * 37) % 300 if b % 7 else 128 * (b % 5) for b in range(n)]
    counts = [b % 4 if b % 5 else 1 for b in range(n)]
    p = ref.Paged4(n, -(-512 // page), 2, dim, page, seed=3)
    for share in (1, 4):
        Q = p.queries(sum(counts), 2 * share, kind)
        ref.check(libgemm, p, Q, counts, lengths)
        ref.check(libgemm, p, Q, counts, lengths, window=50)
        ref.check(libgemm, p, Q, counts, lengths, causal=False)


@pytest.mark.parametrize("n", [1, 2, 7, 40, 113, 150, 229, 300, 520])
def test_pieces_of_every_size(libgemm, n):
    """From less than a tile's opening to some tiles for each block: pieces that
    begin and end inside openings, blocks that get none, tiles in many pieces."""
    dim, page = 64, 128
    lengths = [(b * 331 + n) % 520 if b % 11 else (b * 97) % 8300 for b in range(n)]
    lengths[-1] = 8290
    p = ref.Paged4(min(n, 20), 65, 1, dim, page, seed=n)     # a table too wide for a cluster a tile
    p.table = p.table[torch.arange(n, device="cuda") % 20].contiguous()
    for share in (1, 3):
        ref.check(libgemm, p, p.queries(n, share, torch.bfloat16), [1] * n, lengths)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("share", [1, 8])
def test_bad_indices_in_one_line(libgemm, T, share):
    """Long sequences, whose steps many blocks share: what is out of range is
    skipped and reported, and the other sequences have their results."""
    from accelerator_gb300 import lowbit
    p = ref.Paged4(3, 700, 1, 64, 16)
    Q = p.queries(3 * T, share, torch.float16)
    lengths = [11000, 9000, 10500]
    want = ref.check(libgemm, p, Q, [T] * 3, lengths)
    pages = p.codes[0].shape[0]

    def call(table=p.table, starts=(0, T, 2 * T, 3 * T), at=lengths):
        assert libgemm.debug_status() == libgemm.OK
        O = lowbit.kv_attention(Q, p.cache, table, ints(starts), ints(at))
        assert libgemm.debug_status() == libgemm.ERR_INDEX
        return O

    for bad in (-1, pages, -2 ** 31, 2 ** 31 - 1):
        table = p.table.clone()
        table[1, 300] = bad
        O = call(table=table)
        assert torch.equal(O[:T], want[:T]) and torch.equal(O[2 * T:], want[2 * T:]) and torch.isfinite(O).all()
    for bad in (-1, 700 * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        O = call(at=[11000, bad, 10500])
        assert torch.equal(O[:T], want[:T]) and torch.equal(O[2 * T:], want[2 * T:]) and (O[T:2 * T] == 0).all()
    for starts in ((0, 3 * T + 1, 2 * T, 3 * T), (0, -5, 2 * T, 3 * T), (0, 2 * T, T, 3 * T), (1, T, 2 * T, 3 * T), (0, 0, 0, 0)):
        call(starts=starts)


def test_two_graphs_and_two_streams(libgemm):
    """Graphs of one cache that are replayed in turn and at once, each with its own
    scratch, and calls on two streams."""
    p = ref.Paged4(2, 700, 2, 64, 16)
    calls = [(p.queries(2, 8, torch.float16), [1, 1], [11000, 9000]), (p.queries(140, 8, torch.float16), [70, 70], [3000, 500])]
    want = [p.attend(*c) for c in calls]
    from accelerator_gb300 import lowbit
    from kv_ref import offsets
    args = [(Q, p.cache, p.table, ints(offsets(n)), ints(length)) for Q, n, length in calls]
    graphs, got = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(lowbit.kv_attention(*a))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(5):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for _ in range(5):
        both = [lowbit.kv_attention(*a, stream=s) for a in args for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(both[i], want[i // 2]) for i in range(4))
    assert libgemm.debug_status() == libgemm.OK
