"""The 4-bit cache, the plan of a step and rotary positions on the debug build: a
child process runs every kernel and path on small inputs with each global access
checked against its buffer, compares the results with the release build's, and
finds no bounds report."""
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
from accelerator_gb300 import binding, lowbit, sequences
from kv4_ref import Paged4
from kv_ref import ints, offsets

out = {}
g = torch.Generator(device="cuda").manual_seed(1)

def keep(name, *tensors):
    torch.cuda.synchronize()
    st = binding.debug_status()
    assert st == binding.OK, (name, binding.status_string(st))
    out[name] = [t.cpu() for t in tensors]

def normal(*shape):
    return torch.randn(shape, generator=g, device="cuda")

for dim, page in ((64, 16), (128, 64), (128, 128), (64, 32)):
    p = Paged4(3, -(-2100 // page), 2, dim, page, seed=dim + page)
    for kind in (torch.bfloat16, torch.float16, torch.float32):
        counts, at = [1, 0, 200], [page - 1, 5, 30]
        K, V = normal(201, 2, dim + 1).to(kind), normal(201, 2, dim).to(kind)
        lowbit.kv_append(p.cache, K[:, :, 1:], V, p.table, ints(offsets(counts)), ints(at))
        keep(f"append {dim} {page} {kind}", p.cache.data)
        keep(f"read {dim} {page} {kind}", *lowbit.kv_read(p.cache, p.table, ints(offsets(counts)), ints(at), 201, dtype=kind))
    p.load()
    for name, counts, lengths, share, window in (
            ("decode", [1, 1, 1], [2100, 1, 77], 8, 0), ("few", [2, 0, 3], [900, 5, 60], 3, 0), ("window", [1, 1, 1], [2000, 300, 5], 4, 100),
            ("sixteen", [9, 0, 3], [1000, 5, 60], 2, 0), ("prompt", [300, 70, 1], [700, 70, 900], 4, 0), ("long prompt", [0, 64, 0], [9, 2100, 9], 4, 0)):
        for kind in (torch.bfloat16, torch.float16):
            Q = p.queries(sum(counts), 2 * share, kind)
            keep(f"{name} {dim} {page} {kind}", p.attend(Q, counts, lengths, window=window).float())
# lines of many tiles, and of one long sequence that many blocks share
p = Paged4(40, 30, 4, 64, 16, seed=7)
keep("line", p.attend(p.queries(40, 16, torch.float16), [1] * 40, [1 + 12 * b for b in range(40)]).float())
p = Paged4(1, 700, 1, 64, 16, seed=8)
keep("shared", p.attend(p.queries(1, 4, torch.float16), [1], [11111]).float())
p = Paged4(1, 700, 1, 128, 16, seed=8)
keep("shared by sixteen", p.attend(p.queries(3, 4, torch.bfloat16), [3], [11111]).float())
for n, tokens in ((5, 200), (1500, 4000)):
    L = torch.randint(0, 100, (n,), device="cuda", generator=g).to(torch.int32)
    C = torch.randint(0, 3, (n,), device="cuda", generator=g).to(torch.int32)
    for update in (False, True):
        table = torch.zeros((n, 12), dtype=torch.int32, device="cuda")
        q = sequences.kv_plan(table, L.clone(), C, ints(range(2 * n)), ints([2 * n]), 16, tokens, update=update)
        keep(f"plan {n} {update}", table, *q)
for dim, part in ((64, 64), (128, 32), (33, 30), (1024, 1024)):
    for layout in sequences.LAYOUTS:
        table = sequences.Rotary(part, layout=layout)
        for kind in (torch.bfloat16, torch.float32):
            joint = normal(37, 7, dim).to(kind)
            Q, K = joint[:, :5], joint[:, 5:]
            P = torch.arange(37, device="cuda", dtype=torch.int32) * 1000 - 1000
            q, k = sequences.rotary(Q, K, P, table)
            sequences.rotary(Q, K, P, table, out=(Q, K))
            keep(f"rotary {dim} {layout} {kind}", q[1:].float(), k[1:].float(), joint.float())
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
            if name.split()[0] in ("append", "read", "plan"):
                assert torch.equal(x, y), name
            else:   # the same arithmetic, whose exponentials, sines and sums two compilations may place apart
                assert (x - y).abs().max() <= 0.01 * y.abs().max() + 1e-6, name
