"""Which sources a profile's hash covers: those of its family of kernels."""
import os

import bench

CSRC = os.path.join(bench.ROOT, "row_reduction_norm_gb300", "csrc")
NAMES = [n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h"))]


def read(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return f.read()


def test_a_family_has_its_own_files():
    norm, rope, drop = (bench.family_sources(f, NAMES, read) for f in ("norm", "rope", "dropout"))
    assert {"reg_bf16_res.cu", "rmsnorm_kernels.cuh", "rmsnorm_cluster.cuh", "rmsnorm_tma.cuh", "kernel_pick.cuh"} <= set(norm)
    assert not any(n.startswith(("rope", "drop", "colsum")) for n in norm)
    assert {"rope_kernels.cuh", "rope_ragged.cuh", "rmsnorm_kernels.cuh", "colsum.cu"} <= set(rope)
    assert {"dropout_kernels.cuh", "dropout_shift.cuh", "row_classes.cuh", "rmsnorm_kernels.cuh", "colsum.cu"} <= set(drop)
    assert not any(n.startswith("rope") for n in drop) and not any(n.startswith("drop") for n in rope)
    assert not any(n.endswith("_api.cu") for n in norm + rope + drop)   # choices and checks: no device code


def test_every_kernel_is_in_a_family():
    found = {n for f in bench.KERNEL_FAMILIES for n in bench.family_sources(f, NAMES, read)}
    assert not [n for n in NAMES if n not in found and "__global__" in read(n)]


def test_another_familys_files_do_not_change_a_hash(monkeypatch, tmp_path):
    src = tmp_path / "row_reduction_norm_gb300" / "csrc"
    src.mkdir(parents=True)
    for n in NAMES:
        (src / n).write_text(read(n))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = {f: bench.kernel_source_hash(f) for f in bench.KERNEL_FAMILIES}
    (src / "rope_kernels.cuh").write_text(read("rope_kernels.cuh") + "\nint more;\n")
    (src / "rope_new.cu").write_text("int other;\n")
    after = {f: bench.kernel_source_hash(f) for f in bench.KERNEL_FAMILIES}
    assert after["norm"] == before["norm"] and after["dropout"] == before["dropout"] and after["rope"] != before["rope"]
    (src / "rmsnorm_kernels.cuh").write_text(read("rmsnorm_kernels.cuh") + "\nint more;\n")
    assert all(bench.kernel_source_hash(f) != after[f] for f in after)
