"""The low-bit calls work on the current device: tensors of another one are a
TypeError, before anything is enqueued on a stream that is not theirs."""
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu


def test_tensors_of_another_device(libgemm, monkeypatch):
    from accelerator_gb300 import lowbit
    B, X = torch.randn(64, 32, device="cuda"), torch.ones(2, 64, dtype=torch.float16, device="cuda")
    W = lowbit.w4_quantize(B, 32)
    p = ref.Paged(1, 4, 2, 64, 16)
    K, Q = p.queries(3, 2, torch.float16), p.queries(3, 4, torch.float16)
    starts, first = ref.ints([0, 3]), ref.ints([7])
    calls = [lambda **kw: lowbit.w4_quantize(B, 32, **kw), lambda **kw: lowbit.w4_dequantize(W, **kw),
             lambda **kw: lowbit.gemm_w4(X, W, **kw), lambda **kw: lowbit.kv_append(p.cache, K, K, p.table, starts, first, **kw),
             lambda **kw: lowbit.kv_read(p.cache, p.table, starts, first, 3, **kw),
             lambda **kw: lowbit.kv_attention(Q, p.cache, p.table, starts, ref.ints([10]), **kw)]
    for call in calls:
        call()
    assert libgemm.debug_status() == libgemm.OK
    count = libgemm.launch_count()
    monkeypatch.setattr(lowbit, "_current_device", lambda: 1)     # as it is after torch.cuda.set_device(1)
    for call in calls:
        for kw in ({}, {"stream": torch.cuda.current_stream()}):
            with pytest.raises(TypeError):
                call(**kw)
    assert libgemm.launch_count() == count
