"""The head norm with rotary positions in 64 bits (test side only): the
formulas of the header written out with torch float64, and how far an fp32
evaluation with one rounding may be from them.

Tolerances, u = 2^-24 (half a step of fp32 relative to the value):
  normalised value  18 u relative (the derivation in parity.py: a sum tree of
                    at most 21 levels, mean, eps, rsqrtf, two products; a lane
                    adds at most 8 units, 3 levels in one, 5 shuffles)
  sine and cosine   2e-7 absolute, 3.4 u (the kernels' own series on at most an
                    eighth of a turn: test_rope_angles_host.py)
  rotation          a product and a fused multiply-add: 2 u of |n_a| + |n_b|
so a rotated value is within 24 u (|n_a| + |n_b|), taken as 32 u = 1.9e-6,
and one rounding to the output type, eps / 2 relative.  A value's partner
enters its error, so bounds use m = |n_a| + |n_b| for both.
  gradient of x     g carries 6 u (|dy_a| + |dy_b|); dn = g w one more; the
                    mean of dn x at most 21 + 8 u of the mean of |dn x|; r and
                    r^2 12 u and 24 u; in all under 64 u of
                    r (G |w| + |x| r^2 mean(G |w| |x|)),  G = |dy_a| + |dy_b|
  gradient of w     each term 24 u of G |x| r, and a sum of N terms in any
                    order at most N u of the sum of the terms' sizes
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def pairs_of(head_dim, rot, interleaved):
    """Indices of the first and second element of each rotated pair."""
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def phases(positions, inv_freq, sections):
    """Angles [tokens, pairs] in 64 bits."""
    cols, at = [], 0
    f = inv_freq.double()
    for a, m in enumerate(sections):
        cols.append(positions[a].double()[:, None] * f[None, at:at + m])
        at += m
    return torch.cat(cols, 1)


def rotate(v, theta, head_dim, rot, interleaved, back=False):
    """v [tokens, heads, head_dim] turned by theta; and |a| + |b| of each pair."""
    a, b = pairs_of(head_dim, rot, interleaved)
    c, s = torch.cos(theta)[:, None, :], torch.sin(theta)[:, None, :]
    if back:
        s = -s
    out, size = v.clone(), v.abs()
    out[..., a] = v[..., a] * c - v[..., b] * s
    out[..., b] = v[..., a] * s + v[..., b] * c
    both = v[..., a].abs() + v[..., b].abs()
    size[..., a] = both
    size[..., b] = both
    return out, size


def head_norm(x, w, bias, eps, norm):
    if not norm:
        return x
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r * (1.0 if w is None else w + bias)


def forward(qkv, q, k, d, theta, rot, interleaved, q_w, k_w, eps, bias, norm):
    """(y, bound) in 64 bits for packed rows: the rotated query and key heads."""
    x = qkv[:, :(q + k) * d].double().reshape(-1, q + k, d)
    dbl = lambda w: None if w is None else w.double()
    n = torch.cat((head_norm(x[:, :q], dbl(q_w), bias, eps, norm), head_norm(x[:, q:], dbl(k_w), bias, eps, norm)), 1)
    y, size = rotate(n, theta, d, rot, interleaved)
    return y, 32 * U * size + half_step(qkv.dtype) * (1 + 32 * U) * y.abs()


def backward(dy, qkv, q, k, d, theta, rot, interleaved, q_w, k_w, eps, bias, norm):
    """(dx, bound, dq_w, bound, dk_w, bound); the weights' Nones without weights."""
    t = dy.dtype
    g, size = rotate(dy[:, :(q + k) * d].double().reshape(-1, q + k, d), theta, d, rot, interleaved, back=True)
    if not norm:
        return g, 32 * U * size + half_step(t) * (1 + 32 * U) * g.abs(), None, None, None, None
    x = qkv[:, :(q + k) * d].double().reshape(-1, q + k, d)
    ones = torch.ones(d, dtype=torch.float64, device=x.device)
    wq = ones if q_w is None else q_w.double() + bias
    wk = ones if k_w is None else k_w.double() + bias
    w = torch.cat((wq.expand(q, d), wk.expand(k, d)), 0)[None]
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dn, big = g * w, size * w.abs()
    dx = r * (dn - x * r * r * (dn * x).mean(-1, keepdim=True))
    bound = 64 * U * r * (big + x.abs() * r * r * (big * x.abs()).mean(-1, keepdim=True))
    out = [dx, bound + half_step(t) * (1 + 64 * U) * dx.abs()]
    term, tsize = g * x * r, size * x.abs() * r
    for part in (slice(0, q), slice(q, q + k)):
        dw = term[:, part].sum((0, 1))
        many = term[:, part].shape[0] * term[:, part].shape[1]
        b = (24 + many) * U * tsize[:, part].sum((0, 1))
        out += [dw, b + half_step(t) * dw.abs()] if q_w is not None else [None, None]
    return tuple(out)


def assert_within(got, want, bound, what):
    got = got.double().reshape(want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((off - bound)[bad].max()):.3g} over, "
        f"first at {tuple(int(v) for v in bad.nonzero()[0])}: got {float(got[bad][0])}, want {float(want[bad][0])}")
