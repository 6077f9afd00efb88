"""Queries of zeros and of the smallest numbers over the 4-bit cache: a row of a
padded batch, a head that is switched off."""
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,kind", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("T,share,length", [(1, 1, 300), (1, 4, 20000), (3, 5, 300), (3, 5, 20000), (60, 2, 700)])
def test_rows_of_zeros(libgemm, dim, kind, T, share, length):
    """All scores are 0, so that a row is the mean of the values; rows beside it
    have what they have without it."""
    p = ref.Paged4(2, -(-length // 32), 2, dim, 32, seed=T + share)
    Q = p.queries(2 * T, 2 * share, kind)
    want = ref.check(libgemm, p, Q, [T, T], [length, length // 2])
    empty = torch.zeros(2 * T, 2 * share, dtype=torch.bool, device="cuda")
    empty.view(-1)[::2] = True
    Q[empty] = 0.0
    Q[0, 0] = -0.0
    got = ref.check(libgemm, p, Q, [T, T], [length, length // 2])
    assert torch.equal(got[~empty], want[~empty])
    ref.check(libgemm, p, torch.zeros_like(Q), [T, T], [length, length // 2])


@pytest.mark.parametrize("T", [1, 3, 60])
@pytest.mark.parametrize("exponent", [-133, -127, -126, -116, -115, -114, -113, -112, -111, -100])
def test_rows_of_the_smallest_numbers(libgemm, T, exponent):
    """Down to bfloat16's least, with key scales that bring the scores up again."""
    p = ref.Paged4(1, 10, 2, 128, 32, seed=5)
    Q = torch.sign(p.normal(T, 4, 128)) * 2.0 ** exponent
    ref.check(libgemm, p, Q.to(torch.bfloat16), [T], [300])
    p.scales[0].copy_((p.scales[0].float() * 2.0 ** min(110, -exponent)).to(torch.bfloat16))
    p.load()
    ref.check(libgemm, p, Q.to(torch.bfloat16), [T], [300], scale=2.0 ** -4 * 2.0 ** max(0, -exponent - 110))
