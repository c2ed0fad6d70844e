"""The residual dropout's and the norm gradient's entry points without a GPU:
refusals before any CUDA call, and the tests' generator against the published
vectors of Philox4x32-10 (Salmon et al., SC 2011)."""
import numpy as np
import pytest
import torch

import drop_ref as ref
import row_reduction_norm_gb300 as R
from row_reduction_norm_gb300 import _native as N

P = 1 << 20   # a fake, aligned address: never dereferenced, checks fail first


def fwd(x=P, res=2 * P, w=3 * P, y=4 * P, h=5 * P, rows=4, hidden=64, eps=1e-6, bias=0.0, p=0.1, rng=P, dtype=1):
    return N.rmsnorm_dropout_fwd_status(x, res, w, y, h, rows, hidden, eps, bias, p, rng, dtype)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(res=None), dict(y=None), dict(h=None), dict(y=5 * P), dict(rows=-1), dict(hidden=0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(bias=1.0, w=None), dict(bias=float("inf")), dict(p=-0.1), dict(p=1.0),
    dict(p=float("nan")), dict(p=0.999999), dict(rng=None), dict(rng=P + 4), dict(dtype=2), dict(x=P + 1),
    dict(h=5 * P + 1), dict(rows=1 << 60), dict(w=P + 2, dtype=0),
])
def test_dropout_refusals_without_cuda(over):
    assert fwd(**over) == N.RMSNORM_EINVAL


def test_limits_and_empty_batches_without_cuda():
    assert fwd(hidden=65537) == N.RMSNORM_EUNSUPPORTED
    assert fwd(x=None, res=None, y=None, h=None, rows=0, rng=None) == N.RMSNORM_OK
    assert fwd(rows=0, p=1.5) == N.RMSNORM_EINVAL
    assert bwd(rows=0, dy=None, h=None, dres=None, dx=None, dw=None, w=None) == N.RMSNORM_OK
    assert bwd(hidden=65537) == N.RMSNORM_EUNSUPPORTED
    assert N.load().rmsnorm_bwd_workspace_bytes(4, 65537, 1) == N.RMSNORM_EUNSUPPORTED
    for bad in ((-1, 64, 1), (4, 0, 1), (4, 64, 2)):
        assert N.load().rmsnorm_bwd_workspace_bytes(*bad) == N.RMSNORM_EINVAL


def bwd(dy=P, h=2 * P, w=3 * P, dh=4 * P, dres=5 * P, dx=6 * P, dw=7 * P, rows=4, hidden=64, eps=1e-6, bias=0.0, p=0.1,
        rng=P, dtype=1, ws=None, wb=0):
    return N.rmsnorm_dropout_bwd_status(dy, h, w, dh, dres, dx, dw, rows, hidden, eps, bias, p, rng, dtype, ws, wb)


@pytest.mark.parametrize("over", [
    dict(dy=None), dict(h=None), dict(dres=None), dict(dx=None), dict(dx=5 * P), dict(w=None), dict(w=None, dw=None,
    bias=0.5), dict(p=1.0), dict(p=-1e-3), dict(rng=None), dict(rng=P + 4), dict(dy=P + 1), dict(dh=P + 1),
    dict(dw=7 * P + 1), dict(rows=-1), dict(hidden=-5), dict(eps=float("inf")), dict(dtype=-1),
])
def test_gradient_refusals_without_cuda(over):
    assert bwd(**over) == N.RMSNORM_EINVAL


@pytest.mark.parametrize("over", [dict(dy=None), dict(h=None), dict(dx=None), dict(w=None), dict(eps=-1.0)])
def test_plain_gradient_refusals_without_cuda(over):
    a = dict(dy=P, h=2 * P, w=3 * P, dh=None, dx=5 * P, dw=6 * P, rows=4, hidden=64, eps=1e-6, bias=0.0, dtype=0,
             ws=None, wb=0)
    a.update(over)
    assert N.rmsnorm_bwd_status(*a.values()) == N.RMSNORM_EINVAL


def test_python_calls_refuse_cpu_tensors():
    x = torch.zeros(4, 64)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        R.rms_norm_dropout(x, x, 0.1, rng)
    with pytest.raises(ValueError):
        R.rms_norm_backward(x, x)
    with pytest.raises(ValueError):
        R.rms_norm_dropout_backward(x, x, 0.1, rng)
    with pytest.raises(TypeError):
        R.rms_norm_backward(x.half(), x.half())


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_gives_the_published_vectors(counter, key, want):
    assert ref.philox(np.array(counter, dtype=np.uint64), key).tolist() == list(want)


def test_mask_keeps_what_it_should():
    """400 x 1001 elements at p: the share kept is within five deviations, and
    neither the next offset nor the next seed gives the same mask."""
    for p in (0.05, 0.5, 0.9):
        n = 400 * 1001
        k = ref.kept(400, 1001, p, 12345, 7)
        q = 1 - ref.threshold(p) / 65536
        assert abs(float(k.double().mean()) - q) <= 5 * (q * (1 - q) / n) ** 0.5
        assert not torch.equal(k, ref.kept(400, 1001, p, 12345, 8))
        assert not torch.equal(k, ref.kept(400, 1001, p, 12346, 7))
