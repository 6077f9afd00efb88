"""The first call of each low-bit operator in a process: inside a stream
capture, after any other call on the device, and from many threads at once."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SET_UP = r'''
import sys, threading
sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
import torch
from accelerator_gb300 import binding, lowbit
import kv_ref as ref

A = torch.randn(64, 64, device="cuda")
B, X = torch.randn(200, 96, device="cuda"), torch.randn(3, 200, device="cuda").to(torch.float16)
small, large = ref.Paged(2, 20, 2, 64, 16), ref.Paged(1, 200, 1, 128, 64)     # the large one takes scratch and a joining launch
K, few, many, one = (small.queries(rows, heads, torch.float16) for rows, heads in ((4, 2), (4, 8), (160, 8), (4, 2)))
long = large.queries(1, 4, torch.bfloat16)

def calls():
    W = lowbit.w4_quantize(B, 64)
    lowbit.kv_append(small.cache, K, one, small.table, ref.ints([0, 2, 4]), ref.ints([298, 148]))
    return [lowbit.gemm_w4(X, W), lowbit.w4_dequantize(W), *lowbit.kv_read(small.cache, small.table, ref.ints([0, 2, 4]), ref.ints([298, 148]), 4),
            small.attend(few, [2, 2], [300, 150]), small.attend(many, [80, 80], [300, 150]), large.attend(long, [1], [12000])]

def same(a, b):
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert binding.debug_status() == binding.OK
'''

CAPTURED = SET_UP + r'''
binding.gemm(A, A)                          # the first call on the device
plain = ref.ints
kept = {}
ref.ints = lambda v: kept[str(v)] if str(v) in kept else kept.setdefault(str(v), plain(v))      # made before the capture
for v in ([0, 2, 4], [298, 148], [300, 150], [12000]): ref.ints(v)
for v in ([2, 2], [80, 80], [1]): ref.ints(ref.offsets(v))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
same(got, calls())
'''

THREADS = SET_UP + r'''
found, gate = [None] * 8, threading.Barrier(8)
def work(i):
    q = large.queries(1, 4, torch.bfloat16) if i == 0 else long
    gate.wait()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.default_stream())
    with torch.cuda.stream(stream):
        found[i] = [small.attend(many, [80, 80], [300, 150]), large.attend(long, [1], [12000]), binding.gemm(A, A)]
    stream.synchronize()
torch.cuda.synchronize()
threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]; [t.join() for t in threads]
for f in found[1:]:
    same(f, found[0])
'''


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["captured", "threads"])
def test_first_calls(libgemm, what):
    child = {"captured": CAPTURED, "threads": THREADS}[what]
    r = subprocess.run([sys.executable, "-c", child, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
