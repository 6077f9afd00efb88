"""Attention over pages whose value scales are tiny, zero or orders apart, for
both kernels (few query rows and many): each row against 64 bits, within a
limit that follows from the tokens which that row sees."""
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu

# rows of a sequence x heads to a key head: tiles of 8 and 16 rows, the kernel for many rows
FORMS = [(1, 4), (5, 3), (60, 2)]


@pytest.fixture(params=FORMS, ids=lambda f: f"{f[0]}x{f[1]}")
def form(request):
    return request.param


@pytest.fixture(params=[(64, torch.float16), (128, torch.bfloat16)], ids=["64-fp16", "128-bf16"])
def layout(request):
    return request.param


def paged(form, layout, seed, page=16, width=20):
    (T, share), (dim, kind) = form, layout
    p = ref.Paged(2, width, 2, dim, page, seed=seed)
    return p, [T, T], p.queries(2 * T, 2 * share, kind)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -113, 2.0 ** -120, 2.0 ** -126, 1e-39])
def test_every_value_small(libgemm, form, layout, scale):
    p, counts, Q = paged(form, layout, 1)
    p.vs.fill_(scale)
    ref.check(libgemm, p, Q, counts, [300, 150])


@pytest.mark.parametrize("where", ["first", "last", "all but one"])
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -120, 1e-39, 0.0])
def test_some_values_small(libgemm, form, layout, where, scale):
    """Pages of no weight beside ordinary ones, whatever their codes are."""
    p, counts, Q = paged(form, layout, 2)
    for b, n in enumerate((19, 10)):
        pages = {"first": range(3), "last": range(n - 2, n), "all but one": set(range(n)) - {n // 2}}[where]
        for i in pages:
            p.vs[p.page_of(b, i)] = scale
    ref.check(libgemm, p, Q, counts, [300, 150])


def test_values_as_they_are_appended(libgemm, form, layout):
    """Tokens of 1e-38 (whose page is held as zeros) and of 1e-33, then ordinary ones."""
    from accelerator_gb300 import lowbit
    p, counts, Q = paged(form, layout, 3)
    for n, size in ((20, 1e-38), (20, 1e-33), (260, 1.0)):
        first = ref.ints([at := (0 if n == 20 and size < 1e-35 else 20 if n == 20 else 40)] * 2)
        x = p.normal(2 * n, 2, p.dim)
        lowbit.kv_append(p.cache, x, x * size, p.table, ref.ints([0, n, 2 * n]), first)
        ref.check(libgemm, p, p.queries(2 * min(counts[0], at + n), Q.shape[1], Q.dtype), [min(counts[0], at + n)] * 2, [at + n] * 2)


@pytest.mark.parametrize("ratio", [2.0 ** 20, 2.0 ** 40, 2.0 ** 70])
def test_hidden_pages_of_large_values(libgemm, form, layout, ratio):
    """The last page's values are `ratio` times the others': queries before it
    do not see it, and keep all their bits."""
    p, counts, Q = paged(form, layout, 4)
    T = counts[0]
    lengths = [19 * 16 + min(T, 16) // 2, 9 * 16 + min(T, 16)]
    for b, n in enumerate(lengths):
        p.vs[p.page_of(b, (n - 1) // 16)] *= ratio
    ref.check(libgemm, p, Q, counts, lengths)


@pytest.mark.parametrize("ratio", [2.0 ** 20, 2.0 ** 40, 2.0 ** 70])
def test_pages_of_large_values_before_the_window(libgemm, form, layout, ratio):
    p, counts, Q = paged(form, layout, 5)
    T = counts[0]
    lengths, window = [300, 150], 40
    for b, n in enumerate(lengths):      # the page in which the first query's window begins
        p.vs[p.page_of(b, max(0, n - T - window + 1) // 16)] *= ratio
    ref.check(libgemm, p, Q, counts, lengths, window=window)


@pytest.mark.parametrize("ratio", [2.0 ** 20, 2.0 ** 40, 2.0 ** 60])
@pytest.mark.parametrize("at", [0, 8])
def test_large_values_of_little_weight(libgemm, form, layout, ratio, at):
    """A page of large values that every query sees and gives a weight of about
    1 / ratio: the other pages' part of the result keeps its bits."""
    import math
    p, counts, Q = paged(form, layout, 6)
    Q = torch.ones_like(Q)
    for b in range(2):
        page = p.page_of(b, at)
        p.k[page] = 28                       # every code -100: a score of -sqrt(dim) * 100 * its key scale
        p.ks[page] = math.log(ratio) / (100 * p.dim ** 0.5)
        p.vs[page] = 0.02 * ratio
    ref.check(libgemm, p, Q, counts, [300, 150])


def test_scales_of_any_order(libgemm, form, layout):
    p, counts, Q = paged(form, layout, 7)
    p.vs.copy_(torch.exp2(torch.rand(p.vs.shape, generator=p.g, device="cuda") * 120 - 90))
    p.ks.copy_(torch.exp2(torch.rand(p.vs.shape, generator=p.g, device="cuda") * 12 - 14))
    ref.check(libgemm, p, Q, counts, [300, 150])
    ref.check(libgemm, p, Q, counts, [300, 150], scale=-0.05)
    ref.check(libgemm, p, Q, counts, [300, 150], causal=False)
