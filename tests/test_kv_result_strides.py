"""Strides of attention's result: every (row, head, element) needs a place of
its own; whatever layout gives them one is taken."""
import itertools

import numpy as np
import pytest

from test_kv_cache import FAKE, G, CKv

import ctypes


def attend(libgemm, tokens, q_heads, row, head, dim=64):
    c = CKv(FAKE, FAKE + 4 * G, FAKE + 8 * G, FAKE + 9 * G, 10, 1, 16, dim)
    return libgemm.lib().gemm_kv_attention(ctypes.byref(c), FAKE + 10 * G, q_heads * dim, dim, FAKE + 20 * G, row, head, 1,
                                           q_heads, 0.125, 1, 0, FAKE + 40 * G, 5, FAKE + 41 * G, FAKE + 42 * G, tokens, 1,
                                           None)


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 4), (5, 1), (2, 2), (3, 4), (5, 3), (7, 7)])
def test_results_that_overlap_are_refused(libgemm, tokens, heads):
    import torch
    strides = [0, 1, 32, 63, 64, 65, 96, 128, 130, 192, 200, 256, 300, 320, 448, 500]
    for row, head in itertools.product(strides, strides):
        at = (np.arange(tokens)[:, None, None] * row + np.arange(heads)[None, :, None] * head + np.arange(64)).ravel()
        bad = len(np.unique(at)) < at.size
        if not bad and torch.cuda.is_available():
            continue                                    # would run on the GPU
        rc = attend(libgemm, tokens, heads, row, head)
        want = (libgemm.ERR_INVALID_ARG,) if bad else (libgemm.ERR_CUDA, libgemm.ERR_UNSUPPORTED_DEVICE)
        assert rc in want, (row, head)


@pytest.mark.gpu
def test_an_expanded_result_is_refused(libgemm):
    import torch
    import kv_ref as ref
    p = ref.Paged(1, 4, 2, 64, 16)
    Q = p.queries(3, 4, torch.float16)
    for out in (torch.empty((1, 4, 64), dtype=torch.float16, device="cuda").expand(3, 4, 64),
                torch.empty((3, 1, 64), dtype=torch.float16, device="cuda").expand(3, 4, 64)):
        with pytest.raises(libgemm.GemmError):
            p.attend(Q, [3], [60], out=out)
    by_head = torch.empty((4, 3, 64), dtype=torch.float16, device="cuda").transpose(0, 1)
    assert torch.equal(p.attend(Q, [3], [60], out=by_head), p.attend(Q, [3], [60]))
    assert libgemm.debug_status() == libgemm.OK
