"""A sliding window's pages: those wholly before every row's window may be gone
from the table (a server evicts them), or hold anything."""
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,share", [(1, 4), (5, 3), (60, 2)])
@pytest.mark.parametrize("dim,kind,page", [(64, torch.float16, 16), (128, torch.bfloat16, 32), (128, torch.float16, 128)])
@pytest.mark.parametrize("window", [1, 40, 300])
@pytest.mark.parametrize("gone", ["no page", "past the pool", "nan", "huge"])
def test_pages_before_the_window(libgemm, T, share, dim, kind, page, window, gone):
    lengths = [700, 515]
    p = ref.Paged(2, -(-700 // page), 2, dim, page, seed=window)
    Q = p.queries(2 * T, 2 * share, kind)
    want = ref.check(libgemm, p, Q, [T, T], lengths, window=window)
    for b, n in enumerate(lengths):
        for i in range((n - T - window + 1) // page):        # whole pages before the first row's first token
            if gone in ("nan", "huge"):
                for s in (p.ks, p.vs):
                    s[p.page_of(b, i)] = float("nan") if gone == "nan" else 3e38
            else:
                p.table[b, i] = -1 if gone == "no page" else p.ks.shape[0]
    again = p.attend(Q, [T, T], lengths, window=window)
    assert libgemm.debug_status() == libgemm.OK
    assert torch.equal(again, want)


@pytest.mark.parametrize("T", [1, 60])
def test_a_missing_page_in_the_window_is_reported(libgemm, T):
    p = ref.Paged(1, 40, 1, 64, 16)
    Q = p.queries(T, 2, torch.float16)
    p.table[0, (600 - T - 30 + 1) // 16] = -1                # the page that holds the first row's first token
    p.attend(Q, [T], [600], window=30)
    assert libgemm.debug_status() == libgemm.ERR_INDEX


@pytest.mark.parametrize("T,length", [(1, 20000), (60, 3000)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1, 2 ** 63, 2 ** 64, 2 ** 64 + 5])
def test_a_window_past_every_token_is_none(libgemm, T, length, window):
    """The same result, to the bit: the same split of the tokens, too."""
    p = ref.Paged(1, -(-length // 64), 1, 64, 64)
    Q = p.queries(T, 4, torch.float16)
    want = ref.check(libgemm, p, Q, [T], [length])
    assert torch.equal(p.attend(Q, [T], [length], window=window), want)
    assert libgemm.debug_status() == libgemm.OK
