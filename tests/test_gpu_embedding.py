"""The embedding lookup and its gradient (GB300 only) against their formulas in
64 bits, with the bounds of ends_ref.py."""
import pytest
import torch

import ends_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, std=1.0):
    return torch.empty(shape, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def some_ids(g, n, vocab, kind=torch.int64):
    """Ids of which some lie outside, some come often."""
    ids = torch.randint(-1, vocab + 1, (n,), device=DEV, generator=g)
    often = torch.randint(0, vocab, (1,), device=DEV, generator=g)
    ids = torch.where(torch.rand(n, device=DEV, generator=g) < 0.3, often, ids)
    return ids.to(kind)


WIDTHS = [1, 2, 3, 4, 6, 8, 63, 64, 100, 255, 256, 257, 260, 576, 1001, 2056, 4096]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", WIDTHS)
def test_lookup(width, dtype):
    g = gen(width)
    for n, vocab, scale, kind in ((1, 1, 1.0, torch.int64), (7, 50, 8.0, torch.int32), (1000, 333, 0.3, torch.int64)):
        table = normal(g, vocab, width, dtype=dtype)
        ids = some_ids(g, n, vocab, kind)
        y = R.embedding(ids, table, scale)
        ref.assert_within(y, *ref.embedding(ids, table, scale), f"{n} of {vocab}")
        if scale == 1.0 or scale == 8.0:                       # exact
            assert torch.equal(y.double(), ref.embedding(ids, table, scale)[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width,stride,off", [(64, 72, 0), (64, 65, 0), (64, 64, 1), (96, 100, 2), (40, 44, 4), (5, 9, 3)])
def test_lookup_in_strided_and_unaligned_tables(width, stride, off, dtype):
    g = gen(stride)
    flat = normal(g, 60 * stride + off + 8, dtype=dtype)
    table = flat[off:off + 60 * stride].view(60, stride)[:, :width]
    ids = some_ids(g, 200, 60)
    want = ref.embedding(ids, table, 2.0)[0]
    assert torch.equal(R.embedding(ids, table, 2.0).double(), want)
    room = torch.full((200 * width + 40,), 7.0, dtype=dtype, device=DEV)
    for start in (0, 1, 3, 8):                                 # and into unaligned places, nothing else written
        room.fill_(7.0)
        out = room[start + 8:start + 8 + 200 * width].view(200, width)
        assert R.embedding(ids, table, 2.0, out=out) is out
        assert torch.equal(out.double(), want)
        assert bool((room[:start + 8] == 7.0).all()) and bool((room[start + 8 + 200 * width:] == 7.0).all())


def test_lookup_of_any_shape_and_of_nothing():
    g = gen(1)
    table = normal(g, 20, 33, dtype=BF)
    ids = torch.randint(0, 20, (2, 3, 5), device=DEV, generator=g)
    y = R.embedding(ids, table)
    assert y.shape == (2, 3, 5, 33) and torch.equal(y, table[ids])
    one = R.embedding(torch.tensor(4, device=DEV), table)
    assert torch.equal(one, table[4])
    assert R.embedding(ids[:0], table).shape == (0, 3, 5, 33)
    d = R.embedding_backward(torch.empty(0, 33, dtype=BF, device=DEV), ids.view(-1)[:0], 20)
    assert d.shape == (20, 33) and not d.any()
    kept = table.clone()
    R.embedding_backward(torch.empty(0, 33, dtype=BF, device=DEV), ids.view(-1)[:0], 20, out=table, accumulate=True)
    assert torch.equal(kept, table)


def test_ids_far_outside_and_special_values():
    table = torch.tensor([[float("nan"), float("inf")], [-float("inf"), 1e38], [-0.0, 1e-45]], device=DEV)
    far = [-2 ** 63, 2 ** 63 - 1, 2 ** 32, 2 ** 32 + 1, -1, 3, 0, 1, 2, -2 ** 31]
    y = R.embedding(torch.tensor(far, device=DEV), table, 2.0)
    want = torch.zeros(10, 2, device=DEV)
    want[6:9] = table * 2.0
    ref.assert_within(y, want.double(), torch.zeros_like(want).double(), "far ids")
    near = [i for i in far if -2 ** 31 <= i < 2 ** 31]
    y32 = R.embedding(torch.tensor(near, device=DEV, dtype=torch.int32), table, 2.0)
    ref.assert_within(y32, want[[4, 5, 6, 7, 8, 9]].double(), torch.zeros(6, 2, device=DEV).double(), "near ids")
    d = R.embedding_backward(torch.ones(10, 2, device=DEV), torch.tensor(far, device=DEV), 3)
    assert torch.equal(d, torch.ones(3, 2, device=DEV))


def test_lookup_past_32_bit_offsets():
    vocab, width = 70000, 32776                                # 4.6 GB
    table = torch.zeros(vocab, width, dtype=BF, device=DEV)
    ids = torch.tensor([0, 32767, 65535, 65536, vocab - 1], device=DEV)
    for i, v in enumerate(ids.tolist()):
        table[v, :] = i + 1
        table[v, 7] = -i
    assert torch.equal(R.embedding(ids, table), table[ids])
    dout = table[ids].clone()
    d = R.embedding_backward(dout, ids, vocab, out=table.fill_(3.0))
    assert torch.equal(d[ids], dout) and float(d.float().abs().sum()) == float(dout.float().abs().sum())


# ----------------------------------------------------------------- gradient

@pytest.mark.parametrize("dtype,held", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("width", WIDTHS)
def test_gradient(width, dtype, held):
    g = gen(width)
    for n, vocab, scale in ((1, 1, 1.0), (31, 5, 0.7), (33, 400, 1.0), (700, 90, 3.0)):
        dout, ids = normal(g, n, width, dtype=dtype), some_ids(g, n, vocab, torch.int32 if n == 31 else torch.int64)
        out = torch.full((vocab, width), 5.0, dtype=held, device=DEV)
        d = R.embedding_backward(dout, ids, vocab, scale, out=out)
        assert d is out
        ref.assert_within(d, *ref.embedding_backward(dout, ids, vocab, scale, dtype=held), f"{n} of {vocab}")
        old = normal(g, vocab, width, dtype=held)
        d = R.embedding_backward(dout, ids, vocab, scale, out=old.clone(), accumulate=True)
        ref.assert_within(d, *ref.embedding_backward(dout, ids, vocab, scale, held=old, dtype=held), "added")
        there = torch.zeros(vocab + 1, dtype=torch.bool, device=DEV)
        there[ids.long().where((ids >= 0) & (ids < vocab), vocab)] = True
        assert torch.equal(d[~there[:vocab]], old[~there[:vocab]])     # other rows are left alone


@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 1023, 1024, 50257, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 5])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 1023, 1025, 2048, 2049, 5000, 20000, 70001])
def test_every_token_is_added_once(n, vocab):
    """Whole numbers: sums are exact, so nothing may be lost, doubled or misplaced."""
    g = gen(n + vocab)
    ids = (torch.rand(n, device=DEV, generator=g) ** 6 * vocab).long().clamp(max=vocab - 1)
    ids = torch.where(torch.rand(n, device=DEV, generator=g) < 0.1, -1, ids)
    width = 3
    dout = torch.randint(-8, 9, (n, width), device=DEV, generator=g).float()
    d = R.embedding_backward(dout, ids, vocab, out=torch.full((vocab, width), 9.0, device=DEV))
    assert torch.equal(d.double(), ref.embedding_backward(dout, ids, vocab, 1.0)[0])


@pytest.mark.parametrize("pattern", ["one", "sorted", "falling", "two", "blocks", "none"])
@pytest.mark.parametrize("n", [40, 3000, 33000])
def test_patterns_of_tokens(pattern, n):
    vocab, width = 5000, 264
    i = torch.arange(n, device=DEV)
    ids = {"one": torch.full_like(i, 4321), "sorted": i * vocab // n, "falling": (n - 1 - i) * vocab // n,
           "two": torch.where(i % 3 == 0, 0, vocab - 1), "blocks": i // 45 * 7 % vocab, "none": torch.full_like(i, -1)}[pattern]
    dout = torch.randint(-8, 9, (n, width), device=DEV, generator=gen(n)).to(BF)
    d = R.embedding_backward(dout, ids, vocab, out=torch.full((vocab, width), 9.0, device=DEV))
    assert torch.equal(d.double(), ref.embedding_backward(dout, ids, vocab, 1.0)[0])
    real = normal(gen(n + 1), n, width, dtype=BF)
    ref.assert_within(R.embedding_backward(real, ids, vocab, 0.5), *ref.embedding_backward(real, ids, vocab, 0.5), pattern)


@pytest.mark.parametrize("dtype,held", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("width,stride,off,doff", [(64, 72, 0, 0), (64, 65, 0, 8), (64, 64, 1, 0), (64, 64, 0, 1), (24, 28, 4, 2),
                                                   (6, 9, 3, 5)])
def test_gradient_in_strided_and_unaligned_places(width, stride, off, doff, dtype, held):
    g, n, vocab = gen(off + doff), 500, 77
    flat = torch.full((vocab * stride + off + 16,), 5.0, dtype=held, device=DEV)
    out = flat[off:off + vocab * stride].view(vocab, stride)[:, :width]
    dout = normal(g, n * width + doff, dtype=dtype)[doff:].view(n, width)
    ids = some_ids(g, n, vocab)
    R.embedding_backward(dout, ids, vocab, 1.5, out=out)
    ref.assert_within(out, *ref.embedding_backward(dout, ids, vocab, 1.5, dtype=held), "strided")
    rest = flat.clone()
    rest[off:off + vocab * stride].view(vocab, stride)[:, :width] = 5.0
    assert bool((rest == 5.0).all())


def test_gradient_is_that_of_the_lookup():
    """<dout, lookup(table + e t) - lookup(table)> / e = <gradient, t>: both linear, whole numbers, exact."""
    g, n, vocab, width = gen(3), 300, 40, 24
    whole = lambda *s: torch.randint(-4, 5, s, device=DEV, generator=g).float()
    table, t, dout, ids = whole(vocab, width), whole(vocab, width), whole(n, width), some_ids(g, n, vocab)
    diff = R.embedding(ids, table + t, 2.0) - R.embedding(ids, table, 2.0)
    assert float((diff * dout).double().sum()) == float((R.embedding_backward(dout, ids, vocab, 2.0) * t).double().sum())


def test_the_same_bits_every_time_and_special_values():
    g, n, vocab, width = gen(4), 20000, 3000, 520
    dout, ids = normal(g, n, width, dtype=BF), some_ids(g, n, vocab)
    first = R.embedding_backward(dout, ids, vocab, out=torch.empty(vocab, width, device=DEV))
    for _ in range(3):
        assert torch.equal(first, R.embedding_backward(dout, ids, vocab, out=torch.empty(vocab, width, device=DEV)))
    dout[7], dout[8, 3] = float("nan"), float("inf")
    ids[7], ids[8] = 11, 12
    d = R.embedding_backward(dout, ids, vocab)
    assert bool(d[11].isnan().all()) and float(d[12, 3]) == float("inf")
    clean = torch.ones(vocab, dtype=torch.bool, device=DEV)
    clean[11] = clean[12] = False
    assert bool(d[clean].isfinite().all())


def test_refusals_of_python_calls():
    table, ids = torch.zeros(9, 16, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    dout = torch.zeros(4, 16, device=DEV)
    bad = [lambda: R.embedding(ids.float(), table), lambda: R.embedding(ids.cpu(), table),
           lambda: R.embedding(ids, table.t()), lambda: R.embedding(ids, table, out=torch.zeros(4, 15, device=DEV)),
           lambda: R.embedding(ids, table, out=torch.zeros(4, 16, device=DEV, dtype=BF)),
           lambda: R.embedding(torch.zeros(4, 2, dtype=torch.int64, device=DEV).t(), table),
           lambda: R.embedding_backward(dout, ids[:3], 9), lambda: R.embedding_backward(dout, ids, 0),
           lambda: R.embedding_backward(dout, ids, 9, accumulate=True),
           lambda: R.embedding_backward(dout, ids, 9, out=torch.zeros(8, 16, device=DEV)),
           lambda: R.embedding_backward(dout, ids, 9, out=torch.zeros(9, 16, device=DEV, dtype=BF)),
           lambda: R.embedding_backward(dout, ids, 9, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)),
           lambda: R.embedding_backward(dout.t(), ids, 9)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(R.RmsNormError):
        R.embedding(ids, table, float("inf"))
