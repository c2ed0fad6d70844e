"""The first call of each of these operators in a process captured into a graph,
and made from several threads at once (GB300 only): what a call sets up once a
process or device is set up there."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
import row_reduction_norm_gb300 as R
torch.manual_seed(0)
ids = torch.randint(-1, 900, (70000,), device="cuda")
dout = torch.randint(-4, 5, (70000, 16), device="cuda").float()
logits = torch.randn(40, 60000, device="cuda", dtype=torch.bfloat16)
labels = torch.randint(0, 60000, (40,), device="cuda")
grads = [torch.ones(50000, device="cuda"), torch.ones(7, device="cuda")]
out = [torch.empty_like(g) for g in grads]
ones = torch.ones(40, device="cuda")

def run():
    r = R.token_logprobs(logits, labels, 1.0, 5, True)
    return [R.embedding(ids[:100], dout[:900]), R.embedding_backward(dout, ids, 900), *r,
            R.token_logprobs_backward(logits, labels, r.stats, ones, r.entropy, ones),
            R.clip_grad_norm(grads, 1.0, out=out)]

if MODE == "graph":
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [run()]
    graph.replay()
    torch.cuda.synchronize()
else:
    got = [None] * 6
    go = threading.Barrier(6)
    def one(i):
        s = torch.cuda.Stream()
        go.wait()
        with torch.cuda.stream(s):
            got[i] = run()
        s.synchronize()
    torch.cuda.synchronize()
    out = [torch.empty_like(g) for g in grads]
    threads = [threading.Thread(target=one, args=(i,)) for i in range(6)]
    [t.start() for t in threads]
    [t.join() for t in threads]
want = run()
torch.cuda.synchronize()
for g in got:
    assert g is not None and all(torch.equal(a, b) for a, b in zip(g, want)), [torch.equal(a, b) for a, b in zip(g, want)]
print("fine")
"""


@pytest.mark.parametrize("mode", ["graph", "threads"])
def test_first_calls(mode):
    r = subprocess.run([sys.executable, "-c", f"MODE = {mode!r}\n" + PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr
