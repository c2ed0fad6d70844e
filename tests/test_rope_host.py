"""The rotary and paged-append entry points without a GPU: refusals before any
CUDA call, and a model of the kernel's token lookup on well-formed and
malformed batches (every index it forms stays in bounds)."""
import ctypes
import random

import pytest
import torch

import row_reduction_norm_gb300 as R
from row_reduction_norm_gb300 import _native as N

P = 1 << 20   # a fake, aligned address: never dereferenced, checks fail first


def rope(**over):
    r = N.Rope(P, P, 4, 4, 1, 64, 0)
    r.section[:4] = (32, 0, 0, 0)
    for k, v in over.items():
        if k == "section":
            r.section[:4] = v
        else:
            setattr(r, k, v)
    return r


def fwd(x=P, y=P, tokens=4, xs=768, ys=768, q=8, k=4, d=64, qw=P, kw=P, bias=0.0, eps=1e-6, norm=1, r="default",
        dtype=1):
    return N.rmsnorm_qk_rope_fwd_status(x, y, tokens, xs, ys, q, k, d, qw, kw, bias, eps, norm,
                                        rope() if r == "default" else r, dtype)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(y=None), dict(tokens=-1), dict(xs=767), dict(ys=767), dict(q=-1), dict(q=0, k=0), dict(d=0),
    dict(d=63), dict(qw=None), dict(kw=None), dict(qw=None, kw=None, bias=1.0), dict(bias=float("nan")),
    dict(eps=-1.0), dict(eps=float("inf")), dict(norm=0), dict(norm=2), dict(dtype=2), dict(dtype=-1), dict(r=None),
    dict(x=P + 1), dict(y=P + 1), dict(qw=P + 1), dict(ys=800, y=P, x=P), dict(tokens=1 << 60),
    dict(r=rope(axes=0)), dict(r=rope(axes=5)), dict(r=rope(rot_dim=0)), dict(r=rope(rot_dim=63)),
    dict(r=rope(rot_dim=66, section=(33, 0, 0, 0))), dict(r=rope(section=(31, 0, 0, 0))),
    dict(r=rope(section=(33, -1, 0, 0), axes=2)), dict(r=rope(section=(16, 16, 0, 0))),
    dict(r=rope(axes=2, section=(16, 16, 0, 0), position_stride=3)), dict(r=rope(interleaved=2)),
    dict(r=rope(position_bytes=2)), dict(r=rope(positions=None)), dict(r=rope(inv_freq=None)),
    dict(r=rope(inv_freq=P + 2)), dict(r=rope(positions=P + 4, position_bytes=8)),
])
def test_rope_refusals_without_cuda(over):
    assert fwd(**over) == N.RMSNORM_EINVAL


def test_rope_limits_and_empty_batches_without_cuda():
    assert fwd(d=514, xs=12 * 514, ys=12 * 514) == N.RMSNORM_EUNSUPPORTED
    assert fwd(q=1 << 23, xs=1 << 40, ys=1 << 40) == N.RMSNORM_EUNSUPPORTED
    assert fwd(x=None, y=None, tokens=0) == N.RMSNORM_OK
    assert fwd(x=None, y=None, tokens=0, r=rope(positions=None, inv_freq=None)) == N.RMSNORM_OK
    assert ctypes.sizeof(N.Rope) == 56 and ctypes.sizeof(N.PagedKV) == 112


def bwd(dy=P, x=P, dx=P, tokens=4, gs=768, xs=768, ds=768, q=8, k=4, d=64, qw=P, kw=P, dqw=P, dkw=P, bias=0.0,
        eps=1e-6, norm=1, r="default", dtype=1, ws=P, wb=None):
    wb = 1024 * 2 * 64 * 4 if wb is None else wb
    return N.rmsnorm_qk_rope_bwd_status(dy, x, dx, tokens, gs, xs, ds, q, k, d, qw, kw, dqw, dkw, bias, eps, norm,
                                        rope() if r == "default" else r, dtype, ws, wb)


@pytest.mark.parametrize("over", [
    dict(dy=None), dict(x=None), dict(dx=None), dict(gs=767), dict(xs=767), dict(ds=767), dict(dqw=None),
    dict(dkw=None), dict(qw=None, kw=None), dict(ws=None), dict(ws=P + 8), dict(wb=1024 * 2 * 64 * 4 - 1),
    dict(norm=0), dict(dqw=P + 1), dict(gs=800), dict(xs=800), dict(dy=P + 1), dict(r=rope(positions=None)),
    dict(tokens=-1), dict(d=62, r=rope(rot_dim=64)),
])
def test_rope_gradient_refusals_without_cuda(over):
    assert bwd(**over) == N.RMSNORM_EINVAL


def test_rope_gradient_workspace_bytes():
    assert R.rmsnorm_qk_rope_bwd_workspace_bytes(64) == 1024 * 2 * 64 * 4
    for bad in (0, -2, 63):
        with pytest.raises(N.RmsNormError):
            R.rmsnorm_qk_rope_bwd_workspace_bytes(bad)
    assert N.load().rmsnorm_qk_rope_bwd_workspace_bytes(514) == N.RMSNORM_EUNSUPPORTED


def paged(**over):
    kv = N.PagedKV(P, P, P, P, P, None, 8, 16 * 4 * 64, 4 * 64, 64, 3, 8, 100, 16, 1, 1.0, 1.0)
    for k, v in over.items():
        setattr(kv, k, v)
    return kv


def app(x=P, qo=2 * P, tokens=4, xs=1024, qs=512, q=8, k=4, d=64, qw=P, kw=P, bias=0.0, eps=1e-6, norm=1, r="default",
        kv="default", dtype=1):
    return N.rmsnorm_qkv_append_status(x, qo, tokens, xs, qs, q, k, d, qw, kw, bias, eps, norm,
                                       rope(positions=None) if r == "default" else r,
                                       paged() if kv == "default" else kv, dtype)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(qo=None), dict(k=0), dict(q=-1), dict(xs=1023), dict(qs=511), dict(kv=None), dict(r=None),
    dict(x=P, qo=P), dict(r=rope(positions=None, axes=2, section=(16, 16, 0, 0))),
    dict(kv=paged(cache_dtype=0)), dict(kv=paged(cache_dtype=3)), dict(kv=paged(cache_dtype=2, k_scale=0.0)),
    dict(kv=paged(cache_dtype=2, v_scale=float("nan"))), dict(kv=paged(cache_dtype=2, v_scale=-1.0)),
    dict(kv=paged(cache_dtype=2, k_scale=float("inf"))), dict(kv=paged(seqs=-1)), dict(kv=paged(max_pages=-1)),
    dict(kv=paged(num_pages=-1)), dict(kv=paged(page_size=0)), dict(kv=paged(page_table_stride=7)),
    dict(kv=paged(page_stride=-1)), dict(kv=paged(row_stride=-1)), dict(kv=paged(head_stride=-1)),
    dict(kv=paged(page_stride=1 << 58)), dict(kv=paged(cu_tokens=None)), dict(kv=paged(cache_lens=None)),
    dict(kv=paged(page_table=None)), dict(kv=paged(k_cache=None)), dict(kv=paged(v_cache=None)),
    dict(kv=paged(k_cache=P + 1)), dict(kv=paged(cu_tokens=P + 2)), dict(kv=paged(dropped=P + 2)),
    dict(kv=paged(page_table=None, num_pages=0)),
])
def test_append_refusals_without_cuda(over):
    assert app(**over) == N.RMSNORM_EINVAL


def test_append_empty_batches_without_cuda():
    assert app(x=None, qo=None, tokens=0) == N.RMSNORM_OK
    assert app(kv=paged(seqs=0, cu_tokens=None, cache_lens=None, page_table=None, max_pages=0)) == N.RMSNORM_OK


def test_python_calls_refuse_cpu_tensors():
    x = torch.zeros(4, 12 * 64)
    pos, f = torch.arange(4), torch.ones(32)
    with pytest.raises(ValueError):
        R.qk_norm_rope(x, 8, 4, 64, pos, f)
    with pytest.raises(ValueError):
        R.qk_norm_rope_backward(x, x, 8, 4, 64, pos, f)
    with pytest.raises(ValueError):
        R.qkv_append(x, x, x, x, x, x, 4, 4, 64, f)
    with pytest.raises(TypeError):
        R.qk_norm_rope(x.half(), 8, 4, 64, pos, f)


# ------------------------------------------- model of the kernel's lookup

class Bounded:
    """A list that refuses an index outside it."""

    def __init__(self, v):
        self.v = v

    def __getitem__(self, i):
        assert 0 <= i < len(self.v), f"index {i} of {len(self.v)}"
        return self.v[i]


def sequence_of(cu, seqs, token):
    """The kernel's search."""
    if token < seqs and cu[token] <= token and token < cu[token + 1]:
        return token
    lo, hi = 0, seqs
    while hi - lo > 1:
        mid = lo + (hi - lo) // 2
        if cu[mid] <= token:
            lo = mid
        else:
            hi = mid
    assert 0 <= lo < seqs
    return lo


def cache_row(table, seqs, max_pages, num_pages, page_size, seq, index):
    if index < 0 or index > 0x7FFFFFFF:
        return None
    n = index // page_size
    if n >= max_pages:
        return None
    page = table[seq * max_pages + n]
    if page < 0 or page >= num_pages:
        return None
    return page, index - n * page_size


@pytest.mark.parametrize("seqs", [1, 2, 3, 31, 32, 33, 64, 100, 1023, 1024, 1025, 3000])
def test_lookup_model_finds_every_token(seqs):
    rng = random.Random(seqs)
    for empty in (0.0, 0.5, 0.95):
        cu = [0]
        for _ in range(seqs):
            cu.append(cu[-1] + (0 if rng.random() < empty else rng.randint(1, 5)))
        want = [s for s in range(seqs) for _ in range(cu[s], cu[s + 1])]
        at = range(cu[-1]) if cu[-1] < 400 else rng.sample(range(cu[-1]), 400)
        for t in at:
            assert sequence_of(Bounded(cu), seqs, t) == want[t]


def test_lookup_model_stays_in_bounds_on_malformed_batches():
    rng = random.Random(7)
    odd = [-2 ** 31, -1, 0, 1, 5, 2 ** 31 - 1]
    for _ in range(3000):
        seqs = rng.choice([1, 2, 5, 32, 33, 70])
        cu = Bounded([rng.choice(odd + [rng.randint(0, 100)]) for _ in range(seqs + 1)])
        max_pages, num_pages, page_size = rng.randint(0, 4), rng.randint(0, 6), rng.choice([1, 7, 16, 2 ** 31 - 1])
        table = Bounded([rng.choice(odd) for _ in range(seqs * max_pages)])
        token = rng.randint(0, 120)
        s = sequence_of(cu, seqs, token)
        assert 0 <= s < seqs
        index = rng.choice(odd) + token - cu[s]
        row = cache_row(table, seqs, max_pages, num_pages, page_size, s, index)
        assert row is None or (0 <= row[0] < num_pages and 0 <= row[1] < page_size)
