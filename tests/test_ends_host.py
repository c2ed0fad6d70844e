"""The embedding's, the log probabilities' and the clipping's entry points
without a GPU: refusals before any CUDA call, workspaces, empty calls."""
import ctypes
import math

import pytest
import torch

import row_reduction_norm_gb300 as R
from row_reduction_norm_gb300 import _native as N

P = 1 << 20   # a fake, aligned address: never dereferenced, checks fail first
BAD, MANY, OK = N.RMSNORM_EINVAL, N.RMSNORM_EUNSUPPORTED, N.RMSNORM_OK


def look(tokens=P, size=8, table=2 * P, y=3 * P, count=4, vocab=100, width=64, stride=64, scale=1.0, dtype=1):
    return N.rmsnorm_embedding_fwd_status(tokens, size, table, y, count, vocab, width, stride, scale, dtype)


@pytest.mark.parametrize("over", [
    dict(tokens=None), dict(tokens=P + 4), dict(tokens=P + 2, size=4), dict(size=2), dict(table=None), dict(y=None),
    dict(table=P + 1), dict(y=P + 1), dict(table=P + 2, dtype=0), dict(count=-1), dict(vocab=0), dict(width=0),
    dict(stride=63), dict(scale=math.inf), dict(scale=math.nan), dict(dtype=2), dict(count=1 << 60),
    dict(stride=1 << 60),
])
def test_lookup_refusals(over):
    assert look(**over) == BAD


def test_lookup_limits():
    assert look(width=65537, stride=65537) == MANY
    assert look(count=0, tokens=None, table=None, y=None) == OK
    assert look(count=0, dtype=7) == BAD


def grad(dy=P, tokens=2 * P, size=8, d=3 * P, count=4, vocab=100, width=64, stride=64, scale=1.0, acc=0, dtype=1,
         gd=1, ws=4 * P, wb=1 << 40):
    return N.rmsnorm_embedding_bwd_status(dy, tokens, size, d, count, vocab, width, stride, scale, acc, dtype, gd, ws, wb)


@pytest.mark.parametrize("over", [
    dict(dy=None), dict(dy=P + 1), dict(tokens=None), dict(tokens=P + 4), dict(size=1), dict(d=None), dict(d=P + 1),
    dict(d=P + 2, gd=0), dict(count=-1), dict(vocab=-3), dict(width=0), dict(stride=1), dict(scale=math.nan),
    dict(acc=2), dict(dtype=0, gd=1), dict(dtype=3), dict(gd=2), dict(ws=None), dict(ws=4 * P + 8), dict(wb=0),
])
def test_lookup_gradient_refusals(over):
    assert grad(**over) == BAD


def test_lookup_gradient_limits():
    assert grad(width=65537, stride=65537) == MANY
    assert grad(vocab=(1 << 30) + 1) == MANY
    assert grad(count=(1 << 30) + 1) == MANY
    assert grad(count=0, dy=None, tokens=None, acc=1) == OK
    need = N.rmsnorm_embedding_bwd_workspace_bytes(4, 100, 64)
    assert need > 0 and grad(wb=need - 1) == BAD
    lib = N.load()
    for bad in ((-1, 5, 5), (5, 0, 5), (5, 5, 0)):
        assert lib.rmsnorm_embedding_bwd_workspace_bytes(*bad) == BAD
    assert lib.rmsnorm_embedding_bwd_workspace_bytes(5, 5, 65537) == MANY
    assert lib.rmsnorm_embedding_bwd_workspace_bytes(1 << 30, 1 << 30, 65536) > 0   # nothing overflows


def logp(x=P, tokens=2 * P, size=8, lp=3 * P, stats=4 * P, ent=5 * P, tlp=6 * P, tid=7 * P, rows=4, vocab=100, stride=100,
         top=5, temp=1.0, dtype=1):
    return N.rmsnorm_logprobs_fwd_status(x, tokens, size, lp, stats, ent, tlp, tid, rows, vocab, stride, top, temp, dtype)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(x=P + 1), dict(tokens=None), dict(tokens=P + 4), dict(size=3), dict(lp=P + 2), dict(stats=P + 4),
    dict(ent=P + 1), dict(tlp=None), dict(tid=None), dict(tid=P + 3), dict(rows=-1), dict(vocab=0), dict(stride=99),
    dict(top=-1), dict(top=33), dict(top=6, vocab=5), dict(temp=0.0), dict(temp=-1.0), dict(temp=math.nan),
    dict(temp=math.inf), dict(temp=1e-39), dict(temp=1e38 * 2), dict(dtype=2), dict(stride=1 << 61),
])
def test_logprob_refusals(over):
    assert logp(**over) == BAD


def test_logprob_limits():
    assert logp(vocab=(1 << 20) + 1, stride=1 << 21) == MANY
    assert logp(rows=0, x=None, tokens=None, tlp=None) == OK
    assert logp(rows=0, top=40) == BAD


def dlogp(x=P, tokens=2 * P, size=8, stats=4 * P, g=3 * P, ent=5 * P, h=6 * P, d=7 * P, rows=4, vocab=100, stride=100,
          dstride=100, temp=1.0, dtype=1):
    return N.rmsnorm_logprobs_bwd_status(x, tokens, size, stats, g, ent, h, d, rows, vocab, stride, dstride, temp, dtype)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(tokens=None), dict(stats=None), dict(stats=P + 4), dict(g=P + 1), dict(ent=None), dict(h=P + 2),
    dict(d=None), dict(d=P + 1), dict(dstride=99), dict(stride=1), dict(rows=-1), dict(vocab=0), dict(temp=0.0),
    dict(dtype=-1), dict(dstride=1 << 61),
])
def test_logprob_gradient_refusals(over):
    assert dlogp(**over) == BAD


def test_logprob_gradient_limits():
    assert dlogp(vocab=(1 << 20) + 1, stride=1 << 21, dstride=1 << 21) == MANY
    assert dlogp(rows=0, x=None, stats=None, d=None) == OK


def array(*entries):
    a = (N.Grad * len(entries))()
    for e, (g, o, n, t) in zip(a, entries):
        e.grad, e.out, e.count, e.dtype = g, o, n, t
    return a


@pytest.mark.parametrize("over", [
    dict(grads=None), dict(n=-1), dict(norm=None), dict(norm=P + 2), dict(ws=None), dict(ws=P + 8), dict(wb=64),
    dict(max_norm=-1.0), dict(max_norm=math.nan), dict(grads=array((None, P, 4, 0))),
    dict(grads=array((P, None, 4, 0))), dict(grads=array((P, P, -1, 0))), dict(grads=array((P, P, 4, 2))),
    dict(grads=array((P + 1, P, 4, 1))), dict(grads=array((P, P + 2, 4, 0))),
])
def test_clip_refusals(over):
    a = dict(grads=array((P, P, 4, 0)), n=1, max_norm=1.0, norm=P, ws=P, wb=1 << 30)
    a.update(over)
    assert N.rmsnorm_clip_grads_status(*a.values()) == BAD


def test_clip_entries():
    assert ctypes.sizeof(N.Grad) == 32
    a = array((P, P, 4, 0))
    a[0].reserved = 1
    assert N.rmsnorm_clip_grads_status(a, 1, 1.0, P, P, 1 << 30) == BAD
    assert N.rmsnorm_grad_norm_status(a, 1, P, P, 1 << 30) == BAD
    huge = array((P, P, 1 << 45, 0))
    assert N.rmsnorm_grad_norm_status(huge, 1, P, P, 1 << 30) == MANY
    assert N.rmsnorm_grad_norm_workspace_bytes() > 0


def test_python_calls_refuse_cpu_tensors():
    x, ids = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: R.embedding(ids, x), lambda: R.embedding_backward(x, ids, 10),
                 lambda: R.token_logprobs(x, ids), lambda: R.token_logprobs_backward(x, ids, x, None),
                 lambda: R.grad_norm([x]), lambda: R.clip_grad_norm([x], 1.0), lambda: R.grad_norm([]),
                 lambda: R.clip_grad_norm([None], 1.0), lambda: R.clip_grad_norm([x], 1.0, out=[])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: R.embedding(ids, x.half()), lambda: R.token_logprobs(x.half(), ids),
                 lambda: R.embedding_backward(x.half(), ids, 10)):
        with pytest.raises(TypeError):
            call()
