"""Plans whose counts are more than the step has rows for: sequences get the rows
that there is room for, in their order, and lengths, pages and table follow those
alone, so that later steps go on from what is in the cache."""
import copy
import random

import pytest
import torch

from kv_ref import ints
from test_sequences import plan

pytestmark = pytest.mark.gpu


def cut(counts, tokens):
    """What each sequence gets of `tokens` rows."""
    got = []
    for n in counts:
        got.append(min(n, tokens))
        tokens -= got[-1]
    return got


def old_table(rng, n, width):
    """Rows that others had before: numbers of pages everywhere."""
    return [[rng.randint(0, 5000) for _ in range(width)] for _ in range(n)]


@pytest.mark.parametrize("update", [False, True])
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("n", [1, 3, 33, 257, 1100, 2100])
def test_counts_past_the_room(libgemm, n, page, update):
    from accelerator_gb300 import sequences
    rng = random.Random(n + page)
    for share in (0.0, 0.3, 0.7, 0.999):
        lengths = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, 90)]) for _ in range(n)]
        counts = [rng.choice([0, 1, page, 2 * page + 1, rng.randint(0, 40)]) for _ in range(n)]
        counts[-1] += 1
        tokens = int(share * sum(counts))
        width = -(-max(a + b for a, b in zip(lengths, counts)) // page) + 12 // page + 1
        table = old_table(rng, n, width)
        need = sum(-(-(a + b + 4) // page) for a, b in zip(lengths, counts))
        free = rng.sample(range(10000, 30000 + need), need)
        t, L, A = ints(table), ints(lengths), ints([need])
        assert libgemm.debug_status() == libgemm.OK
        got = sequences.kv_plan(t, L, ints(counts), ints(free), A, page, tokens, update=update)
        assert libgemm.debug_status() == libgemm.ERR_INDEX
        want = plan(table, lengths, cut(counts, tokens), free, need, page, tokens)
        assert t.tolist() == table
        for name, x in want.items():
            assert getattr(got, name).tolist() == x, name
        # the next step, in which all have room, takes pages of its own for what was cut off
        counts, lengths, height = [rng.randint(0, 4) for _ in range(n)], want["lengths"], want["available"][0]
        before = copy.deepcopy(table)
        want = plan(table, lengths, counts, free, height, page, sum(counts))
        got = sequences.kv_plan(t, got.lengths, ints(counts), ints(free), got.available, page, sum(counts), update=update)
        assert libgemm.debug_status() == libgemm.OK
        assert t.tolist() == table
        for name, x in want.items():
            assert getattr(got, name).tolist() == x, name
        # no page has two owners among those that steps took
        taken = [p for old, new in zip(before, table) for p, q in zip(new, old) if p != q]
        assert len(set(taken)) == len(taken)


def test_a_recorded_step_without_room(libgemm):
    """A cut-off sequence's row of the table held another's page before: what is written
    for it in the replays that follow goes to pages of its own."""
    from accelerator_gb300 import lowbit, sequences
    page, heads, dim = 16, 1, 64
    cache = lowbit.Kv4Cache.empty(12, heads, dim, page)
    cache.data.zero_()
    table = ints([[0, 0, 0], [0, 0, 0]])                  # page 0 is sequence 0's; row 1 is reused
    lengths, counts, free, available = ints([5, 0]), ints([1, 20]), ints(range(1, 12)), ints([11])
    K, V = (torch.randn(9, heads, dim, device="cuda").to(torch.bfloat16) for _ in range(2))
    lowbit.kv_append(cache, K[:5], V[:5], table[:1], ints([0, 5]), ints([0]))
    kept = cache.data[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = sequences.kv_plan(table, lengths, counts, free, available, page, 9, update=True)
        lowbit.kv_append(cache, K, V, table, p.starts, p.first)
    graph.replay()                                        # 1 + 8 rows of 1 + 20
    assert libgemm.debug_status() == libgemm.ERR_INDEX
    assert lengths.tolist() == [6, 8] and available.tolist() == [10] and table[1].tolist() == [11, 0, 0]
    counts.copy_(ints([0, 9]))
    graph.replay()                                        # a second page for sequence 1
    assert libgemm.debug_status() == libgemm.OK
    assert lengths.tolist() == [6, 17] and available.tolist() == [9] and table[1].tolist() == [11, 10, 0]
    slots = [11 * page + i for i in range(8, 16)] + [10 * page]
    assert p.slots.tolist() == slots and p.positions.tolist() == list(range(8, 17))
    lowbit.kv_append(cache, K[:1], V[:1], table[:1], ints([0, 1]), ints([5]))
    again = lowbit.Kv4Cache.empty(1, heads, dim, page)
    again.data.copy_(kept[None])
    lowbit.kv_append(again, K[:1], V[:1], table[:1], ints([0, 1]), ints([5]))
    assert torch.equal(cache.data[0], again.data[0])      # sequence 0's page has its own six tokens
    assert libgemm.debug_status() == libgemm.OK
