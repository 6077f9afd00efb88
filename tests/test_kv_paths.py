"""Both attention kernels in every form against 64 bits: tokens shared over
blocks and joined by a second launch, walks of many blocks, signs, windows,
strides, NaN, batches of prompts and single tokens."""
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, torch.float16, 16), (64, torch.bfloat16, 128), (128, torch.bfloat16, 64), (128, torch.float16, 32)]
layouts = pytest.mark.parametrize("dim,kind,page", LAYOUTS)


@layouts
@pytest.mark.parametrize("T,share", [(1, 1), (1, 8), (3, 5)])
@pytest.mark.parametrize("window", [0, 9000])
def test_few_rows_joined_by_a_second_launch(libgemm, dim, kind, page, T, share, window):
    """Few tiles over a table of more than 8192 tokens: one of many shares, one
    of a single one, an empty one, one of a token."""
    counts, lengths = [T, T, T, T, 0], [20011, 130, 0, 1, 500]
    p = ref.Paged(5, -(-20011 // page), 2, dim, page, seed=T + share)
    Q, before = p.queries(4 * T, 2 * share, kind), libgemm.launch_count()
    ref.check(libgemm, p, Q, counts, lengths, window=window)
    assert libgemm.launch_count() == before + 2


@layouts
@pytest.mark.parametrize("counts,lengths", [([300, 0, 41], [3001, 700, 41]), ([1000], [1300]), ([130, 130], [2600, 100])])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 700), (False, 0)])
def test_many_rows_joined_by_a_second_launch(libgemm, dim, kind, page, counts, lengths, causal, window):
    p = ref.Paged(len(counts), -(-max(lengths) // page), 1, dim, page, seed=len(counts))
    Q, before = p.queries(sum(counts), 3, kind), libgemm.launch_count()
    ref.check(libgemm, p, Q, counts, lengths, causal=causal, window=window)
    assert libgemm.launch_count() == before + 2


@layouts
def test_many_rows_over_many_blocks(libgemm, dim, kind, page):
    """Enough tiles that each walks all its blocks itself."""
    counts, lengths = [300, 513, 700, 90], [4000, 2111, 1900, 90]
    p = ref.Paged(4, -(-4000 // page), 8, dim, page)
    Q = p.queries(sum(counts), 16, kind)
    ref.check(libgemm, p, Q, counts, lengths)
    ref.check(libgemm, p, Q, counts, lengths, window=333)


@layouts
@pytest.mark.parametrize("rows", [3, 60, 400])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-6, 2.0])
def test_scales_of_any_sign(libgemm, dim, kind, page, rows, scale):
    p = ref.Paged(1, -(-1500 // page), 2, dim, page)
    ref.check(libgemm, p, p.queries(rows, 4, kind), [rows], [1500], scale=scale)


@layouts
@pytest.mark.parametrize("causal", [True, False])
def test_many_rows_that_see_nothing(libgemm, dim, kind, page, causal):
    counts, lengths = [200, 300, 90], [60, 0, 1]
    p = ref.Paged(3, -(-60 // page), 1, dim, page)
    O = ref.check(libgemm, p, p.queries(590, 2, kind), counts, lengths, causal=causal)
    assert (O[:140] == 0).all() and (O[200:589] == 0).all() and (O[589] != 0).any()


@layouts
@pytest.mark.parametrize("rows,length", [(60, 300), (500, 1500)])      # whole, and joined
def test_strided_rows_and_results(libgemm, dim, kind, page, rows, length):
    p = ref.Paged(1, -(-length // page), 2, dim, page)
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
    """In a query: in its row and head.  In a page's scales: in the rows that see it."""
    p = ref.Paged(1, -(-length // page), 2, dim, page)
    Q = p.queries(rows, 4, kind)
    want = ref.check(libgemm, p, Q, [rows], [length])
    Q[rows // 2, 3, 5] = float("nan")
    got = p.attend(Q, [rows], [length])
    assert torch.isnan(got[rows // 2, 3]).all()
    got[rows // 2, 3] = want[rows // 2, 3]
    assert torch.equal(got, want)
    Q[rows // 2, 3, 5] = 0.5
    want = p.attend(Q, [rows], [length])
    last = (length - 1) // page
    for scales in (p.ks, p.vs):
        kept = scales.clone()
        scales[p.page_of(0, last), 1] = float("nan")
        got = p.attend(Q, [rows], [length])
        hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
        hit[max(0, last * page - (length - rows)):] = True
        assert torch.isnan(got[hit, 2:]).all()
        assert torch.equal(got[~hit], want[~hit]) and torch.equal(got[:, :2], want[:, :2])
        scales.copy_(kept)
    assert libgemm.debug_status() == libgemm.OK


@layouts
@pytest.mark.parametrize("share", [1, 4, 5])
def test_prompts_and_single_tokens_together(libgemm, dim, kind, page, share):
    counts = [1, 1, 700, 1, 0, 1, 1, 33, 1, 1, 1, 2]
    lengths = [900, 17, 700, 1, 300, 0, 513, 40, 1300, 64, 65, 600]
    p = ref.Paged(len(counts), -(-1300 // page), 2, dim, page, seed=share)
    ref.check(libgemm, p, p.queries(sum(counts), 2 * share, kind), counts, lengths)


@layouts
@pytest.mark.parametrize("rows", [1, 5, 60])
def test_the_same_on_every_run(libgemm, dim, kind, page, rows):
    p = ref.Paged(2, -(-12000 // page), 2, dim, page)
    Q = p.queries(2 * rows, 4, kind)
    want = p.attend(Q, [rows, rows], [12000, 5000])
    for _ in range(5):
        assert torch.equal(p.attend(Q, [rows, rows], [12000, 5000]), want)
