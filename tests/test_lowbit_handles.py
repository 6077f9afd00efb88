"""The handles of 4-bit matrices and caches hold addresses and sizes of their
tensors: they cannot be changed under a call's feet."""
import copy

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_cache_is_fixed(libgemm):
    from accelerator_gb300 import lowbit
    cache = lowbit.KvCache.empty(2, 1, 64, 16)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "heads", "head_dim", "page_tokens", "device", "index"):
        held = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, held)
        with pytest.raises(AttributeError):
            delattr(cache, name)
        assert getattr(cache, name) is held
    cache.k_scales.fill_(2.0)                       # contents are the caller's
    assert (cache.k_scales == 2).all()
    with pytest.raises(AttributeError):
        cache.other = 1


def test_matrix_is_fixed(libgemm):
    from accelerator_gb300 import lowbit
    made = lowbit.w4_quantize(torch.randn(64, 32, device="cuda"), 32)
    for W in (made, lowbit.W4Matrix(made.codes.clone(), made.scales.clone(), 64, 32, 32)):
        for name in ("codes", "scales", "K", "N", "group", "device", "index"):
            with pytest.raises(AttributeError):
                setattr(W, name, getattr(W, name))
        assert (W.K, W.N, W.group) == (64, 32, 32)
        lowbit.gemm_w4(torch.ones(2, 64, dtype=torch.float16, device="cuda"), W)


def test_empty_matrix(libgemm):
    from accelerator_gb300 import lowbit
    W = lowbit.w4_quantize(torch.empty((0, 20), device="cuda"), 32)
    assert W.codes.numel() == 0 and W.scales.numel() == 0


def test_copies_have_addresses_of_their_own(libgemm):
    from accelerator_gb300 import lowbit
    W = lowbit.w4_quantize(torch.randn(64, 32, device="cuda"), 32)
    X = torch.ones(2, 64, dtype=torch.float16, device="cuda")
    want = lowbit.gemm_w4(X, W)
    shared, apart = copy.copy(W), copy.deepcopy(W)
    W.codes.fill_(0x88)                             # zeros
    assert (lowbit.gemm_w4(X, shared) == 0).all() and torch.equal(lowbit.gemm_w4(X, apart), want)

    cache = lowbit.KvCache.empty(2, 1, 64, 16)
    table, starts, first = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[1, 0]], [0, 20], [0]))
    x = torch.randn(20, 1, 64, device="cuda")
    lowbit.kv_append(cache, x, x, table, starts, first)
    want = lowbit.kv_read(cache, table, starts, first, 20)
    apart = copy.deepcopy(cache)
    lowbit.kv_append(cache, 0 * x, 0 * x, table, starts, first)
    assert all(torch.equal(a, b) for a, b in zip(lowbit.kv_read(apart, table, starts, first, 20), want))
    assert libgemm.debug_status() == libgemm.OK
