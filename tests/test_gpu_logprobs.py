"""Log probabilities of tokens, entropy, alternatives and their gradient (GB300
only) against their formulas in 64 bits, with the bounds of ends_ref.py."""
import pytest
import torch

import ends_ref as ref
from test_gpu_embedding import BF, DEV, F32, gen, normal

pytestmark = pytest.mark.gpu
LOW = float("-inf")

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R


def check(logits, ids, temperature, top):
    rows, vocab = logits.shape
    r = R.token_logprobs(logits, ids, temperature, top, entropy=True)
    want = ref.Rows(logits, temperature)
    ref.assert_within(r.logprobs, *ref.logprobs(want, ids, vocab), "log probabilities")
    assert torch.equal(r.stats[:, 0].double(), want.m)
    ref.assert_within(r.stats[:, 1], want.log, want.log_bound, "log of the sum")
    ref.assert_within(r.entropy, want.entropy, want.entropy_bound, "entropy")
    if top:
        best = ref.likeliest(logits, top)
        assert torch.equal(r.top_ids.long(), best), "alternatives"
        ref.assert_within(r.top_logprobs, *want.at(best), "their log probabilities")
    return r


def ids_of(g, rows, vocab, kind=torch.int64):
    return torch.randint(-1, vocab + 1, (rows,), device=DEV, generator=g).to(kind)


VOCABS = [1, 2, 7, 8, 9, 33, 100, 255, 256, 1000, 1023, 1024, 1025, 2047, 2048, 2049, 4100, 16383, 16385, 32768, 50257, 131072]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", VOCABS)
def test_rows_of_logits(vocab, dtype):
    g = gen(vocab)
    for rows, temperature, top, kind in ((1, 1.0, min(32, vocab), torch.int64), (3, 0.37, min(20, vocab), torch.int32),
                                         (40, 1.9, min(1, vocab), torch.int64), (200, 1.0, 0, torch.int64)):
        check(normal(g, rows, vocab, dtype=dtype, std=3.0), ids_of(g, rows, vocab, kind), temperature, top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab,stride,off", [(50257, 50257, 0), (50257, 50304, 0), (1001, 1001, 3), (4096, 4097, 1),
                                              (4096, 4104, 8), (300, 305, 7), (16, 17, 5)])
def test_strides_and_alignment(vocab, stride, off, dtype):
    """And the same bits wherever a row lies, and however many there are."""
    g, rows = gen(off), 19
    flat = normal(g, rows * stride + off, dtype=dtype, std=3.0)
    logits = flat[off:off + rows * stride].view(rows, stride)[:, :vocab]
    ids = ids_of(g, rows, vocab)
    r = check(logits, ids, 0.8, 5)
    for many in (1, 2, 300):
        s = R.token_logprobs(logits[3:4].expand(many, vocab).contiguous(), ids[3:4].expand(many).contiguous(), 0.8, 5, True)
        for a, b in zip(r, s):
            assert torch.equal(a[3:4].expand_as(b), b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_row_has_the_same_bits_in_every_batch(dtype):
    g = gen(8)
    for vocab in (2000, 50000, 131072):
        logits, ids = normal(g, 700, vocab, dtype=dtype, std=4.0), torch.randint(0, vocab, (700,), device=DEV, generator=g)
        whole = R.token_logprobs(logits, ids, 1.3, 7, True)
        for a, b in ((0, 1), (1, 3), (5, 30), (100, 260), (650, 700)):
            for x, y in zip(whole, R.token_logprobs(logits[a:b], ids[a:b], 1.3, 7, True)):
                assert torch.equal(x[a:b], y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top", [1, 5, 20, 32])
def test_ties_and_orders(top, dtype):
    """Rows with few values, constant, rising, falling, with both zeros, with all large ones in a place."""
    g, vocab = gen(top), 40000
    i = torch.arange(vocab, device=DEV)
    rows = [torch.zeros(vocab, device=DEV), torch.randint(0, 3, (vocab,), device=DEV, generator=g).float(),
            i.float() * 1e-3, -i.float() * 1e-3, torch.where(i % 2 == 0, 0.0, -0.0), (i % 256).float(),
            torch.where((i >= 4096) & (i < 4096 + 40), 50.0 + i % 7, normal(g, vocab)),
            torch.where(i % 2048 < 8, 9.0, normal(g, vocab)), torch.where(i == vocab - 1, 1.0, LOW),
            torch.where(i >= vocab - 3, 0.0, LOW), torch.where(i < 2, 1.0, LOW)]
    logits = torch.stack(rows).to(dtype)
    check(logits, torch.randint(0, vocab, (len(rows),), device=DEV, generator=g), 1.0, top)
    check(logits[:, :top].contiguous(), torch.zeros(len(rows), dtype=torch.int64, device=DEV), 1.0, top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [5, 3000, 50257])
def test_masks(vocab, dtype):
    g, rows = gen(vocab), 12
    logits = normal(g, rows, vocab, std=3.0)
    share = torch.tensor([0.0, 0.3, 0.9, 0.99, 0.999, 1.0], device=DEV).repeat(2)[:, None]
    hidden = torch.rand(rows, vocab, device=DEV, generator=g) < share
    ids = torch.randint(0, vocab, (rows,), device=DEV, generator=g)
    kept = hidden.scatter(1, ids[:, None], share[:, 0:1] == 1.0)
    kept[6:] = hidden[6:]                                      # in the lower half the token itself may be masked
    check(logits.masked_fill(kept, LOW).to(dtype), ids, 0.9, min(5, vocab))
    # masks of the type's lowest value are numbers like others
    lowest = torch.finfo(dtype).min
    check(logits.to(dtype).masked_fill(kept, lowest), ids, 0.7, min(5, vocab))
    # and a row without any logit: -infinity, no entropy, no gradient
    r = R.token_logprobs(torch.full((2, vocab), LOW, dtype=dtype, device=DEV), ids[:2], 1.0, min(3, vocab), True)
    assert bool((r.logprobs == LOW).all()) and bool((r.entropy == 0).all()) and bool((r.stats == LOW).all())
    assert r.top_ids.tolist() == [list(range(min(3, vocab)))] * 2 and bool((r.top_logprobs == LOW).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_values(dtype):
    vocab = 5000
    big = torch.finfo(dtype).max
    logits = torch.zeros(6, vocab, device=DEV)
    logits[0, 3], logits[1] = big, -big
    logits[2, 4], logits[2, 5] = big, -big
    logits[3] = torch.linspace(-1e4, 1e4, vocab, device=DEV)
    logits[4] = 1e-30
    logits[5, 0] = 88.0
    ids = torch.tensor([3, 7, 4, vocab - 1, 0, 1], device=DEV)
    check(logits.to(dtype), ids, 1.0, 4)
    check(logits.to(dtype), ids, 0.01, 4)
    check(logits.to(dtype), ids, 100.0, 4)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_and_infinity(dtype):
    g, vocab = gen(2), 3000
    logits = normal(g, 5, vocab)
    logits[1, 17] = float("nan")
    logits[2, 2999] = float("inf")
    logits[3] = float("nan")
    ids = torch.tensor([5, 5, 2999, 0, 5], device=DEV)
    r = R.token_logprobs(logits.to(dtype), ids, 1.0, 3, True)
    for i in (1, 2, 3):
        assert bool(r.logprobs[i].isnan()) and bool(r.entropy[i].isnan()) and bool(r.top_logprobs[i].isnan().all())
    assert torch.equal(r.top_ids.long(), ref.likeliest(logits.to(dtype), 3))
    assert bool(r.logprobs[[0, 4]].isfinite().all())
    d = R.token_logprobs_backward(logits.to(dtype), ids, r.stats, torch.ones(5, device=DEV), r.entropy,
                                  torch.ones(5, device=DEV))
    assert bool(d[1].isnan().any()) and bool(d[[0, 4]].isfinite().all())


def test_parts_asked_for():
    g = gen(1)
    logits, ids = normal(g, 9, 700), ids_of(g, 9, 700)
    all_of = R.token_logprobs(logits, ids, 1.0, 3, True)
    none = R.token_logprobs(logits, None)
    assert none.logprobs is None and none.entropy is None and none.top_ids is None and torch.equal(none.stats, all_of.stats)
    only = R.token_logprobs(logits, None, top=3)
    assert torch.equal(only.top_ids, all_of.top_ids) and torch.equal(only.top_logprobs, all_of.top_logprobs)
    assert torch.equal(R.token_logprobs(logits, ids).logprobs, all_of.logprobs)
    empty = R.token_logprobs(logits[:0], ids[:0], top=2, entropy=True)
    assert empty.logprobs.shape == (0,) and empty.top_ids.shape == (0, 2)


# ----------------------------------------------------------------- gradient

def check_gradient(logits, ids, temperature, use_g, use_h, out=None, seed=0):
    g, rows = gen(seed), logits.shape[0]
    r = R.token_logprobs(logits, ids, temperature, 0, True)
    dl = normal(g, rows) if use_g else None
    dh = normal(g, rows) if use_h else None
    if use_g and rows > 2:
        dl[1] = 0.0
    d = R.token_logprobs_backward(logits, ids if use_g else None, r.stats, dl, r.entropy if use_h else None, dh, temperature,
                                  out)
    want = ref.logprobs_backward(logits, ids if use_g else None, r.stats, dl, r.entropy if use_h else None, dh, temperature)
    ref.assert_within(d, *want, f"gradient of {use_g}, {use_h}")
    return d


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", VOCABS)
def test_gradient(vocab, dtype):
    g = gen(vocab)
    for rows, temperature, use_g, use_h in ((1, 1.0, True, True), (5, 0.4, True, False), (33, 1.7, False, True),
                                            (3, 1.0, True, True)):
        logits = normal(g, rows, vocab, dtype=dtype, std=3.0)
        check_gradient(logits, ids_of(g, rows, vocab, torch.int32 if rows == 5 else torch.int64), temperature, use_g, use_h)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab,stride,off,dstride,doff", [
    (50257, 50257, 0, 50257, 0), (1001, 1001, 3, 1001, 3), (4096, 4097, 1, 4096, 0), (4096, 4096, 0, 4097, 1),
    (300, 304, 8, 305, 7), (16, 17, 5, 19, 2), (2052, 2060, 4, 2056, 8)])
def test_gradient_strides_and_alignment(vocab, stride, off, dstride, doff, dtype):
    g, rows = gen(doff), 11
    logits = normal(g, rows * stride + off, dtype=dtype, std=3.0)[off:].view(rows, stride)[:, :vocab]
    flat = torch.full((rows * dstride + doff + 24,), 7.0, dtype=dtype, device=DEV)
    out = flat[doff:doff + rows * dstride].view(rows, dstride)[:, :vocab]
    ids = ids_of(g, rows, vocab)
    d = check_gradient(logits, ids, 0.8, True, True, out)
    assert d is out
    rest = flat.clone()
    rest[doff:doff + rows * dstride].view(rows, dstride)[:, :vocab] = 7.0
    assert bool((rest == 7.0).all())
    assert torch.equal(check_gradient(logits, ids, 0.8, True, True), d.contiguous())   # the same wherever it lies


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_masked_rows_in_place(dtype):
    g, rows, vocab = gen(5), 8, 3001
    logits = normal(g, rows, vocab, std=3.0)
    ids = torch.randint(0, vocab, (rows,), device=DEV, generator=g)
    hidden = torch.rand(rows, vocab, device=DEV, generator=g) < 0.5
    hidden[0, ids[0]] = True                                    # the token itself
    hidden[1] = True                                            # everything
    logits = logits.masked_fill(hidden, LOW).to(dtype)
    ids[2] = -1
    d = check_gradient(logits, ids, 1.2, True, True)
    assert not d[1].any()
    r = R.token_logprobs(logits, ids, 1.2, 0, True)
    ones = torch.ones(rows, device=DEV)
    want = R.token_logprobs_backward(logits, ids, r.stats, ones, r.entropy, ones, 1.2)
    x = logits.clone()
    assert R.token_logprobs_backward(x, ids, r.stats, ones, r.entropy, ones, 1.2, out=x) is x
    assert torch.equal(x, want)
    # rows that nothing reaches are zeros, whatever they hold
    x = logits.clone()
    x[3] = float("nan")
    ones[3] = 0.0
    assert not R.token_logprobs_backward(x, ids, r.stats, ones)[3].any()


def test_gradient_against_differences():
    """Central differences of the formula in 64 bits along random directions:
    off by e^2 / 6 of a third derivative (below 10 |t|^3 here) and the
    gradient's own bound."""
    g, rows, vocab, temperature, e = gen(9), 6, 200, 0.9, 1e-3
    logits, t = normal(g, rows, vocab, std=2.0), normal(g, rows, vocab)
    ids = torch.randint(0, vocab, (rows,), device=DEV, generator=g)
    gl, gh = normal(g, rows), normal(g, rows)

    def value(x):
        r = ref.Rows(x, temperature)
        return r.at(ids[:, None])[0][:, 0] * gl.double() + r.entropy * gh.double()

    diff = (value(logits.double() + e * t.double()) - value(logits.double() - e * t.double())) / (2 * e)
    r = R.token_logprobs(logits, ids, temperature, 0, True)
    d = R.token_logprobs_backward(logits, ids, r.stats, gl, r.entropy, gh, temperature)
    bound = ref.logprobs_backward(logits, ids, r.stats, gl, r.entropy, gh, temperature)[1]
    # stats and entropy are themselves off by their bounds, about 1e-5 of the values
    slack = e * e * 10 * t.double().abs().amax(-1) ** 3 * (gl.abs() + gh.abs()) + 1e-4 * (gl.abs() + gh.abs())
    off = ((d.double() * t.double()).sum(-1) - diff).abs()
    assert bool((off <= (bound * t.double().abs()).sum(-1) + slack).all())


def test_rows_past_32_bit_offsets():
    rows, vocab = 17000, 131072                                 # 4.5 GB
    logits = torch.zeros(rows, vocab, dtype=BF, device=DEV)
    ids = torch.arange(rows, device=DEV) * 7 % vocab
    at = torch.tensor([0, 8191, 8192, 16383, 16384, rows - 1], device=DEV)
    logits[at, ids[at]] = 5.0
    r = R.token_logprobs(logits, ids, 1.0, 2)
    want = ref.Rows(logits[at], 1.0)
    ref.assert_within(r.logprobs[at], *ref.logprobs(want, ids[at], vocab), "far rows")
    assert torch.equal(r.top_ids[at, 0].long(), ids[at])
    g = torch.zeros(rows, device=DEV)
    g[at] = 1.0
    d = R.token_logprobs_backward(logits, ids, r.stats, g, out=logits)
    assert bool((d[at].float().sum(-1).abs() < 0.1).all())
    assert int((d != 0).any(-1).sum()) == len(at)


def test_refusals_of_python_calls():
    x, ids = torch.zeros(4, 64, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    r = R.token_logprobs(x, ids, entropy=True)
    one = torch.ones(4, device=DEV)
    bad = [lambda: R.token_logprobs(x[0], ids), lambda: R.token_logprobs(x.t(), ids), lambda: R.token_logprobs(x, ids[:3]),
           lambda: R.token_logprobs(x, ids.float()), lambda: R.token_logprobs(x, ids.cpu()),
           lambda: R.token_logprobs(x, ids, top=33), lambda: R.token_logprobs(x, ids, top=-1),
           lambda: R.token_logprobs(x[:, :4], ids, top=5),
           lambda: R.token_logprobs_backward(x, ids, r.stats[:3], one),
           lambda: R.token_logprobs_backward(x, None, r.stats, one),
           lambda: R.token_logprobs_backward(x, ids, r.stats, one, None, one),
           lambda: R.token_logprobs_backward(x, ids, r.stats, one.double()),
           lambda: R.token_logprobs_backward(x, ids, r.stats, one, out=torch.zeros(4, 63, device=DEV)),
           lambda: R.token_logprobs_backward(x, ids, r.stats, one, out=torch.zeros(4, 64, device=DEV, dtype=BF))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for t in (0.0, -1.0, float("nan")):
        with pytest.raises(R.RmsNormError):
            R.token_logprobs(x, ids, t)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab,top", [(50000, 20), (131072, 32), (1 << 20, 13)])
def test_more_candidates_than_there_is_room_for(vocab, top, dtype):
    """Groups of threads that see no large logit leave a bound that most of the others' reach: rising, falling, in any order."""
    g = gen(vocab + top)
    i = torch.arange(vocab, device=DEV)
    few = (i // (8 if dtype is BF else 4)) % 32 >= top - 1          # the lanes without
    logits = torch.stack([torch.where(few, -1.0, x) for x in (i * 1e-4, (vocab - i) * 1e-4, normal(g, vocab).abs(),
                                                              (i * 7919 % vocab) * 1e-4)]).to(dtype)
    check(logits, torch.randint(0, vocab, (4,), device=DEV, generator=g), 1.0, top)
