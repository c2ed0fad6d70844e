"""Residual dropout, RMSNorm and their gradients in 64 bits (test side only),
the generator in numpy, and how far an fp32 evaluation may be off.

u = 2^-24.  y from the stored h: 18 u relative (the derivation in parity.py;
a thread's chain here is at most 8 + 8 terms) and a weight bias, taken as
32 u, and one rounding.  Gradient: g one product; mean(g h) at most 29 u of
the mean of |g h|; r and r^2 12 u and 24 u: under 64 u of
r (|g| + |h| r^2 mean |g h|); one more addition for dresidual_out and one
product for the scale.  dw: each term 16 u, and a sum of N terms in any order
at most N u of the sum of the terms' sizes."""
import numpy as np
import torch

from rope_ref import U, half_step


def philox(counter, key):
    """Philox4x32-10 on uint64 arrays that hold 32-bit words: [..., 4], [..., 2]."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k = [int(v) for v in key]
    low, up = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> up) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> up) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1)


def threshold(p):
    return int(np.floor(float(np.float32(p)) * 65536.0 + 0.5))


def kept(rows, hidden, p, seed, offset, first=0):
    """Boolean [rows, hidden], of the rows from `first` on."""
    blocks = (hidden + 7) // 8
    b = np.arange(rows * blocks, dtype=np.uint64) + np.uint64(first * blocks)
    c = np.stack([b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), np.full_like(b, offset & 0xFFFFFFFF),
                  np.full_like(b, (offset >> 32) & 0xFFFFFFFF)], -1)
    w = philox(c, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(rows, blocks * 8)[:, :hidden]
    return torch.from_numpy(u >= np.uint64(threshold(p)))


def forward_h(x, residual, keep, p):
    """residual_out, bit for bit: one fp32 product, one fp32 sum, one rounding."""
    s = torch.tensor(65536.0 / (65536 - threshold(p)), dtype=torch.float32)
    z = torch.where(keep, x.float().cpu() * s, torch.zeros((), dtype=torch.float32))
    return (residual.float().cpu() + z).to(x.dtype)


def norm(h, w, eps, bias):
    """(y, bound) for the stored h."""
    f = h.double()
    y = f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * (w.double() + bias)
    return y, (32 * U + half_step(h.dtype) * (1 + 32 * U)) * y.abs()


def backward(dy, h, w, dh, keep, p, eps, bias):
    """(dresidual, bound, dx, bound, dw, bound)."""
    f, g0 = h.double(), dy.double()
    r = 1.0 / torch.sqrt((f * f).mean(-1, keepdim=True) + eps)
    g = g0 if w is None else g0 * (w.double() + bias)
    d = r * (g - f * r * r * (g * f).mean(-1, keepdim=True))
    size = r * (g.abs() + f.abs() * r * r * (g * f).abs().mean(-1, keepdim=True))
    if dh is not None:
        d = d + dh.double()
        size = size + d.abs() / 64
    bound = 64 * U * size
    step = half_step(dy.dtype) * (1 + 64 * U)
    out = [d, bound + step * d.abs(), None, None, None, None]
    if keep is not None:
        s = 65536.0 / (65536 - threshold(p))
        dx = d * s * keep
        out[2:4] = [dx, (bound * s + 2 * U * dx.abs()) * keep + step * dx.abs()]
    if w is not None:
        terms = g0 * f * r
        dw = terms.sum(0)
        out[4:6] = [dw, (16 + len(terms)) * U * terms.abs().sum(0) + step * dw.abs()]
    return out
