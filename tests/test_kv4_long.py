"""Long contexts of which one block has whole tiles: the error of a sum over all
tokens does not grow with their number as that of its terms' magnitudes would."""
import pytest
import torch

import kv4_ref as ref
from kv_ref import U, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,kind", [(64, torch.float16), (128, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("share", [1, 4, 16])
def test_sums_over_many_tokens(libgemm, dim, kind, share):
    """Keys of zeros, so that all weights are alike and a row is the mean of c s.  The
    largest s of any 16 tokens is 1, so that weights times s, eight bits, enter
    the product as they are.  What is lost, by the way the sums are made:
      two products of 16 tokens for each step of 32, whose sums reach 16 times the
      step's scales: 2^-22 of that each;
      a warp's n / 64 products, and 64 steps to join the parts: 2^-22 each of what the
      sum has so far without the codes' 8;
      the weights' sum, the division and the power of two: 2^-20 of the result, which
      is rounded once."""
    from accelerator_gb300 import lowbit
    n, batch, page = 131072, 512, 64
    p = ref.Paged4(1, n // page, 1, dim, page, seed=share, spare=0)
    p.codes[0].zero_()
    s = torch.rand(p.scales[1].shape, generator=p.g, device="cuda").clamp_(2.0 ** -7, 1.0).to(torch.bfloat16)
    s[..., ::16] = 1.0
    p.scales[1].copy_(s)
    p.load()
    order = p.table[0].long()
    c, s = (x[order].double().transpose(0, 1).reshape(n, -1) for x in (p.codes[1], p.scales[1]))
    v = c * s
    want = v.mean(0)
    warps = v.view(-1, 4, 32, dim).transpose(0, 1).reshape(4, -1, dim).cumsum(1)      # each warp's tokens in its order
    peak = (warps.amax((0, 1)) - warps.amin((0, 1))) / n                              # a piece may begin anywhere
    limit = 2 * 2.0 ** -22 * 16 * s.mean() + (n / 64 + 64) * 2.0 ** -22 * peak + (U[kind] + 2.0 ** -20) * want.abs() + 2.0 ** -25
    Q = p.queries(batch, share, kind)
    table, starts = p.table.expand(batch, -1).contiguous(), torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    got = lowbit.kv_attention(Q, p.cache, table, starts, ints([n] * batch))
    assert libgemm.debug_status() == libgemm.OK
    worst = ((got.double() - want).abs() / limit).max().item()
    assert worst <= 1, worst
