"""The rotary kernels' sine and cosine (sincos_turns, csrc/rope_kernels.cuh),
step by step in numpy: fp32 with fused multiply-adds, against 64 bits.

What they are off by, u = 2^-24.  The angle t is at most an eighth of a turn,
pi / 4, and carries 3 u of itself: an integer rounded to fp32, the constant 2 pi /
2^32, their product.  The sine's and the cosine's derivatives times t are at most
0.56 there, so that is 1.7 u.  The series' own roundings: half a step of the
result, and of its other terms, t^3 / 6 or t^2 / 2, under 3 u, so 1.3 u.  The series'
remainder is 2e-9 and the dropped 2^-33 of a turn 8e-10.  In all under 3.2 u,
1.9e-7; bounds take 2e-7."""
import re

import numpy as np

from row_reduction_norm_gb300 import build as B

F = np.float32


def fma(a, b, c):
    """Rounded twice, to 64 bits and to 32: off by 2^-29 of a step more."""
    return F(a.astype(np.float64) * np.float64(b) + np.float64(c))


def sincos_turns(t32):
    """Of t32 (uint32) times 2^-32 turns."""
    t32 = t32.astype(np.uint32)
    q = (t32 + np.uint32(0x20000000)) >> np.uint32(30)
    t = F((t32 - (q << np.uint32(30))).astype(np.int32)) * F(1.46291807926715968e-9)
    z = t * t
    sr = fma(z, F(2.75573192e-6), F(-1.98412698e-4))
    sr = fma(z, sr, F(8.33333333e-3))
    sr = fma(z, sr, F(-1.66666667e-1))
    sr = fma(t * z, sr, t)
    cr = fma(z, F(-2.75573192e-7), F(2.48015873e-5))
    for c in (-1.38888889e-3, 4.16666667e-2, -0.5, 1.0):
        cr = fma(z, cr, F(c))
    odd = (q & 1).astype(bool)
    s, c = np.where(odd, cr, sr), np.where(odd, sr, cr)
    return np.where(q & 2, -s, s), np.where((q + 1) & 2, -c, c)


def test_the_steps_are_the_kernels():
    src = open(f"{B.CSRC}/rope_kernels.cuh").read()
    body = src[src.index("void sincos_turns"):]
    body = body[:body.index("\n}")]
    numbers = {float(n) for n in re.findall(r"(-?\d\.\d+(?:e-\d+)?)f", body)}
    assert {1.46291807926715968e-9, 2.75573192e-6, -1.98412698e-4, 8.33333333e-3, -1.66666667e-1, -2.75573192e-7,
            2.48015873e-5, -1.38888889e-3, 4.16666667e-2, -0.5} <= numbers


def test_sine_and_cosine_are_within_the_bound():
    rng = np.random.default_rng(1)
    t = np.concatenate([rng.integers(0, 1 << 32, 1 << 20), np.arange(0, 1 << 32, 1 << 14),
                        *[(np.arange(-2000, 2000) + (k << 29)) % (1 << 32) for k in range(8)], np.arange(5000)])
    s, c = sincos_turns(t)
    angle = t.astype(np.float64) * (2 * np.pi / 2 ** 32)
    assert np.abs(s - np.sin(angle)).max() <= 1.99e-7 and np.abs(c - np.cos(angle)).max() <= 1.99e-7
