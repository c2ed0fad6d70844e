"""The native Python calls beside other Python threads (GB300 only): what they
call may block (a launch queue that is full, memory that is allocated), so
other threads have to run meanwhile."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

from test_gpu_limits import calls

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from row_reduction_norm_gb300 import api

# in place of the C ABI's launching functions: arguments are not looked at
SLOW = r"""
#include <unistd.h>
int slow(void) { usleep(150000); return 0; }
"""


def test_other_threads_run_during_a_native_call(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("gcc not installed")
    src, so = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text(SLOW)
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    calls(3)   # everything is loaded
    torch.cuda.synchronize()
    slow = ctypes.cast(ctypes.CDLL(str(so)).slow, ctypes.c_void_p).value
    fast, lib = api._bind_fast(), api.N.load()
    real = [ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in api._FAST_NAMES]
    stamps, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            stamps.append(time.perf_counter())
            time.sleep(0.001)

    t = threading.Thread(target=tick)
    t.start()
    try:
        fast.bind(*(a if "bytes" in n else slow for a, n in zip(real, api._FAST_NAMES)))
        first = time.perf_counter()
        calls(3)   # its six native calls take 150 ms each
        last = time.perf_counter()
    finally:
        fast.bind(*real)
        stop.set()
        t.join()
    assert last - first >= 6 * 0.15
    seen = [s for s in stamps if first <= s <= last]
    gap = max(b - a for a, b in zip([first, *seen], [*seen, last]))
    assert gap < 0.1, f"another thread stood still for {gap * 1e3:.0f} ms"


def test_without_the_native_calls(monkeypatch):
    """The Python bodies on the current stream make the same calls."""
    want = calls(7)
    monkeypatch.setattr(api, "_fast", api._PythonCalls())
    got = calls(7)
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
