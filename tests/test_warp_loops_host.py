"""Loops of the kernels that a warp goes round together, read as text: what
decides whether it goes on is one lane's reading where other warps may change it
meanwhile.  Lanes that read it each for themselves may part, and the shuffles
inside would wait for those that left."""
import os
import re

from row_reduction_norm_gb300 import build as B

SOURCES = [n for n in sorted(os.listdir(B.CSRC)) if n.endswith((".cu", ".cuh"))]


def header_of(text, at):
    """What stands in the brackets that open behind text[at]."""
    start = text.index("(", at)
    depth = 0
    for i in range(start, len(text)):
        depth += (text[i] == "(") - (text[i] == ")")
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("brackets do not close")


def volatile_decisions(text):
    """The conditions of loops and branches that read changing memory."""
    text = re.sub(r"//[^\n]*", "", text)
    heads = (header_of(text, m.end()) for m in re.finditer(r"\b(for|while|if)\b(?= ?\()", text))
    return [h for h in heads if "volatile" in h]


def test_one_lane_reads_what_a_warps_loop_goes_by():
    found = {n: volatile_decisions(open(os.path.join(B.CSRC, n), encoding="utf-8").read()) for n in SOURCES}
    assert len(found["logprobs_kernels.cuh"]) == 1          # the gathering of alternatives
    for name, heads in found.items():
        for h in heads:
            assert re.match(r"\(__shfl_sync\(0xffffffffu, .*, 0\) ", h), f"{name}: {h}"
