"""The low-bit operators on the debug build: a child process runs every kernel
and path on small inputs with each global access checked against its buffer,
compares the results with the release build's, and finds no bounds report."""
import os
import subprocess
import sys

import pytest

from accelerator_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
import torch
from accelerator_gb300 import binding, lowbit
from test_kv_cache import Pool, ints, offsets

out = {}
g = torch.Generator(device="cuda").manual_seed(1)

def keep(name, *tensors):
    torch.cuda.synchronize()
    st = binding.debug_status()
    assert st == binding.OK, (name, binding.status_string(st))
    out[name] = [t.cpu() for t in tensors]

for K, N, dt, group in ((300, 77, torch.float32, 32), (129, 256, torch.bfloat16, 128), (64, 16, torch.float16, 64)):
    B = torch.randn(K, N, device="cuda", generator=g).to(dt)
    W = lowbit.w4_quantize(B, group)
    keep(f"w4 {K} {N}", W.codes, W.scales.float(), lowbit.w4_dequantize(W, dtype=dt).float())
    for M, xt in ((1, torch.bfloat16), (5, torch.float16), (16, torch.bfloat16), (40, torch.float16)):
        X = torch.randn(M, K + 3, device="cuda", generator=g).to(xt)
        for pad in (0, 3):
            x = X[:, :K] if pad else X[:, :K].contiguous()
            keep(f"product {K} {N} {M} {pad}", lowbit.gemm_w4(x, W, dtype=torch.float32))
for dim, page in ((64, 16), (128, 64), (128, 128)):
    pool = Pool(3, -(-2100 // page), 2, dim, page, seed=dim + page)
    table = ints(pool.table)
    for kind in ("bf16", "fp32"):
        counts, at = [1, 0, 200], [page - 1, 5, 30]
        K, V = pool.rows(201, 2, kind), pool.rows(201, 2, kind)
        lowbit.kv_append(pool.gpu, K, V, table, ints(offsets(counts)), ints(at))
        keep(f"append {dim} {page} {kind}", pool.gpu.k_codes, pool.gpu.v_codes, pool.gpu.k_scales, pool.gpu.v_scales)
        keep(f"read {dim} {page} {kind}", *lowbit.kv_read(pool.gpu, table, ints(offsets(counts)), ints(at), 201, dtype=torch.float32))
    for name, counts, lengths, share, window in (("decode", [1, 1, 1], [2100, 1, 77], 8, 0), ("few", [2, 0, 3], [900, 5, 60], 3, 0),
                                                 ("window", [1, 1, 1], [2000, 300, 5], 4, 100), ("prompt", [300, 70, 1], [700, 70, 900], 4, 0),
                                                 ("long prompt", [0, 64, 0], [9, 2100, 9], 4, 0)):
        for kind in ("bf16", "fp16"):
            Q = pool.rows(sum(counts), 2 * share, kind)
            keep(f"{name} {dim} {page} {kind}", lowbit.kv_attention(Q, pool.gpu, table, ints(offsets(counts)), ints(lengths), window=window).float())
# one sequence over a long cache: shared over many blocks and joined by a second launch
pool = Pool(1, 700, 1, 64, 16, seed=7)
Q = pool.rows(1, 4, "fp16")
keep("split", lowbit.kv_attention(Q, pool.gpu, ints(pool.table), ints([0, 1]), ints([11111])).float())
torch.save(out, sys.argv[2])
print("debug" if binding.debug_build() else "release", len(out))
'''


def _child(path, debug):
    env = dict(os.environ, LIBGEMM_DEBUG="1" if debug else "0")
    build.build(debug=debug)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, str(path)], env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert r.stdout.startswith("debug" if debug else "release")


@pytest.mark.gpu
def test_every_path_in_bounds_and_the_same(tmp_path):
    import torch
    for debug in (True, False):
        _child(tmp_path / f"{debug}.pt", debug)
    a, b = (torch.load(tmp_path / f"{debug}.pt") for debug in (True, False))
    assert a.keys() == b.keys()
    for name in a:
        for x, y in zip(a[name], b[name]):
            if name.split()[0] in ("w4", "append", "read"):
                assert torch.equal(x, y), name
            else:   # the same arithmetic, whose exponentials and sums two compilations may place apart
                assert (x - y).abs().max() <= 0.01 * y.abs().max() + 1e-6, name
