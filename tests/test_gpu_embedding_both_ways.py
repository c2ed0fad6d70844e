"""The embedding's gradient without a sort and with one, of the same tokens
(GB300 only).  Tokens are added up without a sort while the square of their
number, times the row's tiles of 256 columns, is at most 2^20: 1024 tokens of up
to 256 columns are, 1025 are not."""
import pytest
import torch

from test_gpu_embedding import BF, DEV, F32, gen

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R


@pytest.mark.parametrize("dtype,held", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("vocab", [3, 50, 5000])
@pytest.mark.parametrize("width", [5, 64, 256])
def test_the_same_sums_without_a_sort_and_with_one(width, vocab, dtype, held):
    """Whole numbers of up to 8, 1024 of them: every sum is exact in fp32, and both ways round it alike."""
    g = gen(width + vocab)
    ids = torch.randint(-1, vocab + 1, (1025,), device=DEV, generator=g)
    ids[-1] = -1                                               # the one more is padding
    dout = torch.randint(-8, 9, (1025, width), device=DEV, generator=g).to(dtype)
    out = [torch.full((vocab, width), 3.0, dtype=held, device=DEV) for _ in range(2)]
    for add in (False, True):
        a = R.embedding_backward(dout[:-1], ids[:-1].contiguous(), vocab, out=out[0], accumulate=add)
        b = R.embedding_backward(dout, ids, vocab, out=out[1], accumulate=add)
        assert torch.equal(a, b)
