"""A process whose first calls of the dense side are captured ones, one after the other in one graph, and then made from
several host threads at once: nothing that is set up once may need a call before."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys, threading
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import linear_ref as R
import speculative_decoding_verification_59_gb300 as sv
sizes = [(1, 1000, 4096), (20, 1000, 4096), (64, 700, 2048), (100, 300, 400), (65, 3000, 2064), (128, 128, 2064), (600, 2000, 16400), (250, 4000, 12304)]
problems = [R.problem(i, *s) for i, s in enumerate(sizes)]
x, xs, w, ws = problems[0]
odd = torch.zeros(33, device="cuda")[1:].view(1, 32)
odd.copy_(xs)
rows = torch.randn((70, 512), device="cuda").to(torch.bfloat16)
torch.cuda.synchronize()

def run():
    out = [t for p in problems for t in (sv.matmul_e4m3(*p), sv.matmul_e4m3(*p, dtype=torch.float32))]
    out.append(sv.matmul_e4m3(x, odd, w, ws))
    out += [sv.add_norm(rows), *sv.add_norm(rows, None, rows, e4m3=True), sv.gated_act(rows), *sv.quantize_e4m3(rows)]
    return out + list(sv.quantize_e4m3(rows, block_rows=128))

def same(a, b):
    return all(torch.equal(s.contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)) for s, t in zip(a, b))

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = run()
graph.replay()
torch.cuda.synchronize()
kept = [t.clone() for t in held]
assert same(kept, run())
results, streams = [None] * 4, [torch.cuda.Stream() for _ in range(4)]

def work(i):
    with torch.cuda.stream(streams[i]):
        for _ in range(5):
            results[i] = run()
threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert all(same(kept, r) for r in results)
print("as before")
"""


def test_first_calls_captured_then_from_threads():
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", CODE.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as before" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
