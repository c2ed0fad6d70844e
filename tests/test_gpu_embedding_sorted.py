"""The embedding's gradient of more tokens than are added up without a sort
(GB300 only): what test_gpu_embedding.py checks for few, with the same bounds."""
import pytest
import torch

import ends_ref as ref
from test_gpu_embedding import BF, DEV, F32, WIDTHS, gen, normal, some_ids

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R


@pytest.mark.parametrize("dtype,held", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("width", WIDTHS)
def test_gradient_and_sums_onto_one(width, dtype, held):
    g, n, vocab, scale = gen(width), 2500, 900, 0.7
    dout, ids = normal(g, n, width, dtype=dtype), some_ids(g, n, vocab)
    d = R.embedding_backward(dout, ids, vocab, scale, out=torch.full((vocab, width), 5.0, dtype=held, device=DEV))
    ref.assert_within(d, *ref.embedding_backward(dout, ids, vocab, scale, dtype=held), "overwritten")
    old = normal(g, vocab, width, dtype=held)
    d = R.embedding_backward(dout, ids, vocab, scale, out=old.clone(), accumulate=True)
    ref.assert_within(d, *ref.embedding_backward(dout, ids, vocab, scale, held=old, dtype=held), "added")
    there = torch.zeros(vocab + 1, dtype=torch.bool, device=DEV)
    there[ids.where((ids >= 0) & (ids < vocab), vocab)] = True
    assert torch.equal(d[~there[:vocab]], old[~there[:vocab]])


@pytest.mark.parametrize("dtype,held", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("width,stride,off,doff", [(64, 72, 0, 0), (64, 65, 0, 8), (64, 64, 1, 0), (64, 64, 0, 1), (24, 28, 4, 2),
                                                   (6, 9, 3, 5), (300, 301, 7, 3)])
def test_strided_and_unaligned_places(width, stride, off, doff, dtype, held):
    g, n, vocab = gen(off + doff), 3000, 177
    flat = torch.full((vocab * stride + off + 16,), 5.0, dtype=held, device=DEV)
    out = flat[off:off + vocab * stride].view(vocab, stride)[:, :width]
    dout = normal(g, n * width + doff, dtype=dtype)[doff:].view(n, width)
    ids = some_ids(g, n, vocab)
    R.embedding_backward(dout, ids, vocab, 1.5, out=out)
    ref.assert_within(out, *ref.embedding_backward(dout, ids, vocab, 1.5, dtype=held), "strided")
    rest = flat.clone()
    rest[off:off + vocab * stride].view(vocab, stride)[:, :width] = 5.0
    assert bool((rest == 5.0).all())


def test_a_table_larger_than_what_is_zeroed_beside_the_sort():
    """And rows of all kinds in it: 3 GB, the last row past 32-bit offsets of bytes."""
    g, n, vocab, width = gen(1), 3000, 400000, 2048
    ids = torch.cat((torch.randint(0, vocab, (n - 4,), device=DEV, generator=g),
                     torch.tensor([0, vocab - 1, vocab, -1], device=DEV)))
    dout = torch.randint(1, 9, (n, width), device=DEV, generator=g).float()
    d = R.embedding_backward(dout, ids, vocab, out=torch.full((vocab, width), 7.0, device=DEV))
    held, at = torch.unique(ids[(ids >= 0) & (ids < vocab)], return_inverse=True)
    want = torch.zeros(len(held), width, device=DEV).index_add_(0, at, dout[(ids >= 0) & (ids < vocab)])
    assert torch.equal(d[held], want)
    assert float(d.sum(dtype=torch.float64)) == float(want.sum(dtype=torch.float64)) and float(d.min()) >= 0.0
    assert int((d != 0).any(-1).sum()) == len(held)


@pytest.mark.parametrize("n,vocab", [(150000, 3000), (300001, 1 << 21), (1 << 20, 500)])
def test_more_tokens_than_the_sort_keeps_in_registers(n, vocab):
    g, width = gen(n), 5
    ids = (torch.rand(n, device=DEV, generator=g) ** 3 * vocab).long()
    dout = torch.randint(-4, 5, (n, width), device=DEV, generator=g).to(BF)
    d = R.embedding_backward(dout, ids, vocab, out=torch.empty(vocab, width, device=DEV))
    assert torch.equal(d.double(), ref.embedding_backward(dout, ids, vocab, 1.0)[0])


def test_the_same_ids_in_both_ways_of_adding_up():
    """1024 tokens are added up without a sort, one more with one: whole numbers, the same sums."""
    g, vocab, width = gen(6), 50, 264
    ids = torch.randint(0, vocab, (1025,), device=DEV, generator=g)
    ids[-1] = -1
    dout = torch.randint(-8, 9, (1025, width), device=DEV, generator=g).float()
    assert torch.equal(R.embedding_backward(dout, ids, vocab), R.embedding_backward(dout[:-1], ids[:-1], vocab))


@pytest.mark.parametrize("n,width", [(1024, 256), (1025, 256), (724, 512), (725, 512), (512, 1024), (513, 1000), (129, 16384),
                                     (64, 65536), (65, 65530)])
def test_few_tokens_of_wide_rows(n, width):
    """Both sides of where the sort begins, which is earlier the wider the rows: whole numbers, the exact sums."""
    g, vocab = gen(n), 40
    ids = some_ids(g, n, vocab)
    dout = torch.randint(-4, 5, (n, width), device=DEV, generator=g).to(BF)
    d = R.embedding_backward(dout, ids, vocab, out=torch.empty(vocab, width, device=DEV))
    assert torch.equal(d.double(), ref.embedding_backward(dout, ids, vocab, 1.0)[0])


@pytest.mark.parametrize("n", [15000, 29184, 29185, 60000, 116736, 233472, 240000])
@pytest.mark.parametrize("vocab", [60, 20000])
def test_shares_of_a_warp_from_a_few_tokens_to_64(n, vocab):
    """Runs of an id that end in a warp's first 32 tokens, in its last ones, and go on: whole numbers, the exact sums."""
    g, width = gen(n + vocab), 11
    ids = torch.randint(-1, vocab, (n,), device=DEV, generator=g)
    dout = torch.randint(-4, 5, (n, width), device=DEV, generator=g).to(BF)
    d = R.embedding_backward(dout, ids, vocab, out=torch.empty(vocab, width, device=DEV))
    assert torch.equal(d.double(), ref.embedding_backward(dout, ids, vocab, 1.0)[0])
