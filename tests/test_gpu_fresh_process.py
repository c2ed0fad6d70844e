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
