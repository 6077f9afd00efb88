"""Rotary positions of tensors that require a gradient: refused where autograd would
lose it, and the forward and backward of a Function."""
import types

import pytest
import torch

from kv_ref import ints


def test_gradients_are_not_lost():
    """(Refused before anything else of the tensors is looked at: no GPU needed.)"""
    from accelerator_gb300 import sequences
    table = types.SimpleNamespace(index=-1, device="cpu", rotary_dim=8)
    Q, K = torch.zeros(2, 3, 8), torch.zeros(2, 1, 8)
    leaf, at = torch.zeros(2, 3, 8, requires_grad=True), torch.zeros(1, dtype=torch.int32)
    for args, out in (((leaf, K), None), ((leaf * 2, None), None), ((K, leaf), None), ((Q, K), (leaf, K)), ((Q, None), (leaf, None))):
        with pytest.raises(TypeError, match="autograd"):
            sequences.rotary(*args, at, table, out=out)
        with torch.no_grad(), pytest.raises(ValueError, match="positions"):      # the next check
            sequences.rotary(*args, at, table, out=out)
    with pytest.raises(ValueError, match="positions"):
        sequences.rotary(Q, K, at, table)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_a_function(libgemm, layout):
    from accelerator_gb300 import sequences
    from test_sequences import turned
    table, positions = sequences.Rotary(32, layout=layout), ints([0, 1, 5, 77, 1000])

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k):
            return sequences.rotary(q, k, positions, table)

        @staticmethod
        def backward(ctx, dq, dk):
            return sequences.rotary(dq.contiguous(), dk.contiguous(), positions, table, inverse=True)

    leaves = [torch.randn(5, h, 40, device="cuda", requires_grad=True) for h in (4, 2)]
    weights = [torch.randn(5, h, 40, device="cuda") for h in (4, 2)]
    with pytest.raises(TypeError):
        sequences.rotary(*leaves, positions, table)
    sum((x * w).sum() for x, w in zip(Turn.apply(*leaves), weights)).backward()
    for x, w in zip(leaves, weights):
        exact = x.detach().double().requires_grad_()
        (turned(exact, positions, table) * w).sum().backward()
        # sines and cosines by 5, two products and a sum by 3 roundings of (|a| + |b|)
        assert (x.grad.double() - exact.grad).abs().max() <= 2 * 8 * 2.0 ** -24 * w.abs().max()
    with torch.no_grad():
        got = sequences.rotary(*leaves, positions, table)
    assert all(torch.equal(a, b) for a, b in zip(got, sequences.rotary(*(x.detach() for x in leaves), positions, table)))
    assert libgemm.debug_status() == libgemm.OK
