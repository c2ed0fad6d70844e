"""The operators at the two ends of a model in 64 bits (test side only):
embedding lookup and its gradient, log probabilities with entropy and
alternatives and their gradient, the norm of many tensors and their clipping;
and how far an fp32 evaluation with one rounding may be from them.

Tolerances, u = 2^-24 (half a step of fp32 relative to the value):
  lookup         a product (u) and the rounding to the output type
  its gradient   n terms in any order: n u of the sum of their sizes; the scale
                 u, adding to what is held u of both, and the rounding
  exponentials   z = (x - m) log2(e) / T carries a subtraction, the factor's own
                 rounding and a product, 3 u |z|; ex2.approx is good to 2^-22,
                 4 u; so a term of the sum is off by (3 |z| + 4) u.  In the
                 combination of units d = (m' - m) log2(e) / T is part of |z|
                 and another ex2 adds 4 u
  their sum      in a lane at most 32 terms, 6 levels to the warp's sum, then
                 units / 32 units a lane and 5 levels: with E|z| the mean of
                 |z| (natural log) under p,  r = (52 + units / 32 + 4 E|z|) u
  its log        r absolute, and logf, 2 u |L|
  log prob.      3 u |z| + that + u |value|
  entropy        L - sum(e z) / s: a term e z is off by (3 |z| + 8) u of itself,
                 their sum as above: 4 u E(z^2) + (60 + units / 32) u E|z|, and
                 r E|z| for the division; 2 u of the result
  its gradient   log p: 3 u |z| + 2 u (|z| + |L|); p another 4 u; a + b log p and
                 the products 6 u more: with w = |g| + |h| (|log p| + |H|)
                 p w (12 + 7 |z| + 4 |L|) u / T, the token's own g: 2 u |g| / T,
                 and the rounding.  Below 2^-126 a p is 0.
  norm           squares u, 8 + 3 levels in a thread, u for sums of sums (kept
                 in two parts): 13 u, half of it for the root, u for its
                 rounding: 8 u.  Clipped: 8 u + 2 u and the rounding
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half of the smallest step there is: results that underflow are off by as much."""
    return 2.0 ** -134 if dtype is torch.bfloat16 else 2.0 ** -150


def rounding(y, dtype):
    return half_step(dtype) * y.abs() + smallest(dtype)


def embedding(ids, table, scale):
    v = table.shape[0]
    there = ((ids >= 0) & (ids < v))[..., None]
    y = torch.where(there, table.double()[ids.long().clamp(0, v - 1)] * scale, 0.0)
    return y, U * y.abs() + rounding(y, table.dtype) * (1 + U)


def embedding_backward(dout, ids, vocab, scale, held=None, dtype=None):
    width = dout.shape[-1]
    d, ids = dout.double().reshape(-1, width), ids.long().reshape(-1)
    there = (ids >= 0) & (ids < vocab)
    d, ids = d[there], ids[there]
    zero = torch.zeros(vocab, width, dtype=torch.float64, device=d.device)
    total = zero.index_put((ids,), d, accumulate=True) * scale
    sizes = zero.index_put((ids,), d.abs(), accumulate=True) * abs(scale)
    n = torch.bincount(ids, minlength=vocab)[:, None]
    bound = (n + 2) * U * sizes
    if held is not None:
        total = total + held.double()
        bound = bound + U * (held.double().abs() + sizes)
    return total, bound + rounding(total, dtype or dout.dtype) * (1 + U)


def unit_of(dtype):
    """Logits of a unit, which the order of a row's sums goes by."""
    return 2048 if dtype is torch.bfloat16 else 1024


class Rows:
    """All that is said of rows of logits, with bounds."""

    def __init__(self, logits, temperature):
        x = logits.double()
        low = float("-inf")
        self.m = x.amax(-1)
        self.none = self.m == low
        base = torch.where(self.none, 0.0, self.m)[:, None]
        self.z = (x - base) / temperature
        e = self.z.exp()
        s = e.sum(-1)
        self.p = torch.where(self.none[:, None], 0.0, e / s[:, None])
        self.log = torch.where(self.none, low, s.log())
        size = torch.where(self.p > 0, self.z.abs(), 0.0)
        mean, square = (self.p * size).sum(-1), (self.p * size * size).sum(-1)
        units = -(-logits.shape[-1] // unit_of(logits.dtype))
        r = (52 + units / 32 + 4 * mean) * U
        self.log_bound = torch.where(self.none, 0.0, r + 2 * U * self.log.abs())
        self.entropy = torch.where(self.none, 0.0, self.log + mean)
        self.entropy_bound = (self.log_bound + 4 * U * square + (60 + units / 32) * U * mean + r * mean
                              + 2 * U * self.entropy.abs())

    def at(self, ids):
        """Log probabilities of [rows, k] ids in the vocabulary."""
        low = float("-inf")
        z = self.z.gather(1, ids.long())
        lp = torch.where(self.none[:, None], low, z - self.log[:, None])
        bound = 3 * U * z.abs() + self.log_bound[:, None] + U * lp.abs()
        return lp, torch.where(lp == low, 0.0, bound)


def logprobs(rows, ids, vocab):
    there = (ids >= 0) & (ids < vocab)
    lp, bound = rows.at(ids.long().clamp(0, vocab - 1)[:, None])
    return torch.where(there, lp[:, 0], 0.0), torch.where(there, bound[:, 0], 0.0)


def likeliest(logits, top):
    """Ids of the largest, ties to the lowest id, NaN as -infinity."""
    x = torch.nan_to_num(logits.double(), nan=float("-inf"), posinf=float("inf"), neginf=float("-inf")) + 0.0
    return torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]


def logprobs_backward(logits, ids, stats, g, entropy, h, temperature):
    """From the stats and the entropy that are given, as the kernel does."""
    x, low = logits.double(), float("-inf")
    rows, vocab = x.shape
    m, log = stats[:, :1].double(), stats[:, 1:].double()
    none = m == low
    z = (x - torch.where(none, 0.0, m)) / temperature
    lp = torch.where(none, low, z - torch.where(none, 0.0, log))
    p = lp.exp()
    there = torch.zeros(rows, dtype=torch.bool, device=x.device) if ids is None else (ids >= 0) & (ids < vocab)
    g = torch.zeros(rows, dtype=torch.float64, device=x.device) if g is None else torch.where(there, g.double(), 0.0)
    h = torch.zeros_like(g) if h is None else h.double()
    ent = torch.zeros_like(g) if entropy is None else entropy.double()
    g = torch.where(none[:, 0], 0.0, g)[:, None]
    onto = torch.zeros_like(x)
    if ids is not None:
        onto.scatter_(1, ids.long().clamp(0, vocab - 1)[:, None], there.double()[:, None])
    flat = torch.where(p > 0, lp, 0.0)
    d = g * (onto - p) - h[:, None] * p * (flat + ent[:, None])
    d = d / temperature
    w = g.abs() + h.abs()[:, None] * (flat.abs() + ent.abs()[:, None])
    size = torch.where(p > 0, z.abs(), 0.0)
    bound = p * w * (12 + 7 * size + torch.where(none, 0.0, 4 * log.abs())) * U + 2 * U * g.abs() * onto + 2.0 ** -125 * w
    return d, bound / temperature + rounding(d, logits.dtype) * (1 + U)


def norm(grads):
    total = sum(float(g.double().square().sum()) for g in grads)
    return total ** 0.5


def clipped(g, n, max_norm):
    f = 1.0 if n <= max_norm else max_norm / n
    y = g.double() * f
    return y, 10 * U * y.abs() + rounding(y, g.dtype) * (1 + 10 * U)


def assert_within(got, want, bound, what):
    # What rounds to nearest beyond the largest fp32 number, (2 - 2^-23) 2^127, is
    # infinite from half a step above it on, (2 - 2^-24) 2^127: such a result
    # (a masked token's z over a temperature below 1) is infinity in fp32.
    want = torch.where(want.abs() >= (2 - 2.0 ** -24) * 2.0 ** 127, want.sign() * float("inf"), want)
    got = got.double().reshape(want.shape)
    same = (got == want) | (got.isnan() & want.isnan())      # infinities and NaN too
    off = (got - want).abs()
    bad = ~(same | (off <= bound))
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {tuple(int(v) for v in bad.nonzero()[0])}: "
        f"got {float(got[bad][0])!r}, want {float(want[bad][0])!r} within {float(bound.expand_as(want)[bad][0]):.3g}")
