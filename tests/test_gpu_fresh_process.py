"""Calls that are the first of their kind in a process (GB300 only): what a
kernel has to be opted in to must not hang on an earlier, larger call."""
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
import torch
import row_reduction_norm_gb300 as R
rows, hidden, dtype, p = 3, int(sys.argv[1]), getattr(torch, sys.argv[2]), float(sys.argv[3])
g = torch.Generator(device="cuda"); g.manual_seed(1)
dy, h = (torch.empty(rows * hidden + 1, device="cuda").normal_(generator=g).to(dtype)[1:].view(rows, hidden) for _ in range(2))
if sys.argv[4] == "aligned":
    dy, h = dy.clone(), h.clone()
w = torch.ones(hidden, device="cuda", dtype=dtype)
if p:
    d, _, dw = R.rms_norm_dropout_backward(dy, h, p, torch.tensor([1, 2], device="cuda"), w)
else:
    d, dw = R.rms_norm_backward(dy, h, w)
f, g0 = h.double(), dy.double()
r = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + 1e-6)
want = r * (g0 - f * r * r * (g0 * f).mean(-1, keepdim=True))
tol = {torch.float32: 1e-5, torch.bfloat16: 1e-2}[dtype]
assert float((d.double() - want).norm() / want.norm()) < tol
assert float((dw.double() - (g0 * f * r).sum(0)).norm() / (g0 * f * r).sum(0).norm()) < tol
print("fine")
"""


# fp32 sums of the columns, and with dropout a mask, of nearly 48 KB and of exactly that
@pytest.mark.parametrize("hidden,dtype,p,place", [(12288, "float32", 0.0, "aligned"), (12200, "float32", 0.0, "aligned"),
                                                  (12161, "float32", 0.0, "off"), (11904, "float32", 0.1, "aligned"),
                                                  (12288, "bfloat16", 0.0, "off"), (11800, "bfloat16", 0.1, "off")])
def test_two_pass_gradient_first(hidden, dtype, p, place):
    """Norms of the errors: fp32 arithmetic within 1e-5, bf16 outputs within a rounding (2^-8) and some."""
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(hidden), dtype, str(p), place], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-800:]


CAPTURED = """
import threading
import torch
from test_gpu_limits import calls
from test_gpu_rope import inputs, normal
import row_reduction_norm_gb300 as R

# a captured step that is the process's first call of every operator
g, qkv, pos, f, qw, kw = inputs("bf16", 40, 4, 2, 64, 64, (32,), 3, extra=2)
dy = normal(g, 40, 6 * 64, dtype=torch.bfloat16)
x, res, dn, dh = (normal(g, 50, 1001, dtype=torch.bfloat16) for _ in range(4))
w = normal(g, 1001, dtype=torch.bfloat16, mean=1.0)
rng = torch.tensor([3, 3], dtype=torch.int64, device="cuda")
kc, vc = (torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
k8, v8 = (torch.zeros(4, 16, 2, 64, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
table, cu, lens = ints(2, 0, 1, 3).view(2, 2), ints(0, 21, 40), ints(5, 0)

def step():
    y, h = R.rms_norm_dropout(x, res, 0.1, rng, w)
    return [R.qk_norm_rope(qkv, 4, 2, 64, pos, f, qw, kw), *R.qk_norm_rope_backward(dy, qkv, 4, 2, 64, pos, f, qw, kw),
            R.qkv_append(qkv, kc, vc, table, cu, lens, 4, 2, 64, f, q_w=qw, k_w=kw),
            R.qkv_append(qkv, k8, v8, table, cu, lens, 4, 2, 64, f, q_w=qw, k_w=kw, k_scale=0.05, v_scale=0.03), y, h,
            *R.rms_norm_dropout_backward(dn, h, 0.1, rng, w, dh), *R.rms_norm_backward(dn, h, w, dh)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, step()):
    assert torch.equal(a, b)
print("fine")
"""

THREADS = """
import threading
import torch
from test_gpu_limits import calls

torch.zeros(1, device="cuda")
got, start = {}, threading.Barrier(4)

def work(i):
    start.wait()
    with torch.cuda.stream(torch.cuda.Stream()):
        got[i] = calls(5)
        torch.cuda.current_stream().synchronize()

threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
assert len(got) == 4
want = calls(5)
torch.cuda.synchronize()
for one in got.values():
    assert all(torch.equal(a, b) for a, b in zip(one, want))
print("fine")
"""


@pytest.mark.parametrize("program", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls(program):
    """Captured into a graph without a call before it; from four threads at once."""
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path.insert(0, 'tests')\n" + program], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-1500:]
