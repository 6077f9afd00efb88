"""Row offsets that do not ascend: reported by every call on a cache, whatever
the rest of the batch, and nothing outside of the arrays is read or written."""
import random

import pytest
import torch

import kv_ref as ref

gpu = pytest.mark.gpu


def lookup(starts, first, rows, log2):
    """(unit, sequence, page of the sequence) of a cache write's units, as the
    kernels find them from the offsets: sequence q's units begin at starts[q] /
    page + 2 q, a search by 32 lanes at a time."""
    n = len(first)
    at = lambda b: max(0, min(rows, starts[b]))             # noqa: E731
    value = lambda b: (at(b) >> log2) + 2 * b               # noqa: E731
    for u in range((rows >> log2) + 2 * n):
        q, hi = 0, n
        while hi - q > 1:
            step = -(-(hi - q) // 32)
            below = sum(q + lane * step < hi and value(q + lane * step) <= u for lane in range(32))
            q, hi = q + max(below - 1, 0) * step, min(hi, q + max(below - 1, 0) * step + step)
        if 0 <= starts[q] <= starts[q + 1] <= rows:
            count, block = starts[q + 1] - starts[q], (first[q] >> log2) + u - value(q)
            if count and first[q] >> log2 <= block and block << log2 < first[q] + count:
                yield u, q, block


def test_units_stay_in_their_sequence():
    """No unit is given a page before its sequence's first or past its last,
    and no two units the same page, for any offsets."""
    rng = random.Random(1)
    for _ in range(3000):
        n, rows = rng.randint(1, 40), rng.randint(1, 300)
        starts = [0] + [rng.randint(0, rows) for _ in range(n - 1)] + [rows]
        if rng.random() < 0.3:
            starts.sort()
        first = [rng.randint(0, 40) for _ in range(n)]
        units = list(lookup(starts, first, rows, 4))
        assert len({(q, block) for _, q, block in units}) == len(units)
        for _, q, block in units:
            assert first[q] >> 4 <= block <= (first[q] + starts[q + 1] - starts[q] - 1) >> 4
        if starts == sorted(starts):
            assert sum(1 for _ in units) == sum(-(-(f + e - s) // 16) - f // 16 for f, s, e in zip(first, starts, starts[1:]) if e > s)


BAD = [[0, 100, 40, 60, 200, 240], [0, 240, 16, 32, 48, 240], [0, 0, 200, 100, 240, 240], [0, 30, 20, 10, 5, 240],
       [5, 10, 20, 30, 40, 240], [0, 10, 20, 30, 40, 239], [0, 10, 20, -30, 40, 240], [0, 10, 20, 400, 40, 240]]


@gpu
@pytest.mark.parametrize("starts", BAD, ids=str)
@pytest.mark.parametrize("share", [1, 8])       # of 48 rows on average, so both kernels
def test_offsets_that_descend_are_reported(libgemm, starts, share):
    from accelerator_gb300 import lowbit
    p = ref.Paged(5, 20, 1, 64, 16)
    K = p.queries(240, 1, torch.float16)
    at, first = ref.ints(starts), ref.ints([0, 3, 30, 0, 17])
    for call in (lambda: lowbit.kv_append(p.cache, K, K, p.table, at, first),
                 lambda: lowbit.kv_read(p.cache, p.table, at, first, 240),
                 lambda: lowbit.kv_attention(p.queries(240, share, torch.float16), p.cache, p.table, at, ref.ints([300] * 5))):
        assert libgemm.debug_status() == libgemm.OK
        call()
        assert libgemm.debug_status() == libgemm.ERR_INDEX
