"""Alternatives of rows that hold many NaN (GB300 only): a NaN counts as
-infinity among them, in rows of one warp, of a block and of a cluster."""
import pytest
import torch

import ends_ref as ref
from test_gpu_embedding import BF, DEV, F32, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R

NAN, LOW = float("nan"), float("-inf")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(640, 1000), (640, 20000), (12, 131072), (5, 2000)])
def test_alternatives_among_many_nan(rows, vocab, dtype):
    g = gen(vocab)
    x = normal(g, rows, vocab, std=3.0)
    share = torch.tensor([0.0, 0.1, 0.5, 0.9, 0.999, 1.0], device=DEV).repeat(rows // 6 + 1)[:rows, None]
    hidden = torch.rand(rows, vocab, device=DEV, generator=g) < share
    x = torch.where(hidden, NAN, x)
    x[rows // 2:] = torch.where((x[rows // 2:] < 0), LOW, x[rows // 2:])     # masks too, whose NaN tie with them
    logits = x.to(dtype)
    clean = ~hidden.any(-1)
    ids = torch.randint(0, vocab, (rows,), device=DEV, generator=g)
    for top in (1, 5, 20, 32):
        r = R.token_logprobs(logits, ids, 0.8, top, True)
        assert torch.equal(r.top_ids.long(), ref.likeliest(logits, top)), top
        assert bool(r.top_logprobs[~clean].isnan().all()) and bool(r.logprobs[~clean].isnan().all())
        want = ref.Rows(logits[clean], 0.8)
        ref.assert_within(r.top_logprobs[clean], *want.at(r.top_ids[clean]), "rows without NaN")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(640, 2000), (640, 20000), (3, 131072)])
def test_nan_beside_groups_that_hold_the_largest(rows, vocab, dtype):
    """Lanes of NaN beside lanes of rising, falling and equal logits: the first bound is one that nearly all others reach."""
    i = torch.arange(vocab, device=DEV)
    for top in (5, 20, 32):
        few = (i // (8 if dtype is BF else 4)) % 32 >= top - 1
        kinds = [torch.where(few, NAN, y) for y in (i * 1e-3, (vocab - i) * 1e-3, torch.ones(vocab, device=DEV))]
        logits = torch.stack(kinds).repeat(rows // 3 + 1, 1)[:rows].to(dtype)
        r = R.token_logprobs(logits, None, top=top)
        assert torch.equal(r.top_ids.long(), ref.likeliest(logits, top)), top


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1, 9, 3000, 50257])
def test_everything_of_a_row_with_nan_or_infinity_is_nan(vocab, dtype):
    """And its gradient; the rows beside it are as without it."""
    g = gen(vocab)
    x = normal(g, 7, vocab)
    x[1, vocab // 2] = NAN
    x[2, vocab - 1] = float("inf")
    x[3] = NAN
    x[4] = LOW
    x[5] = torch.where(torch.arange(vocab, device=DEV) == 0, NAN, LOW)
    logits, ids, one = x.to(dtype), torch.zeros(7, dtype=torch.int64, device=DEV), torch.ones(7, device=DEV)
    r = R.token_logprobs(logits, ids, 1.0, min(3, vocab), True)
    d = R.token_logprobs_backward(logits, ids, r.stats, one, r.entropy, one)
    for part in (r.logprobs, r.stats, r.entropy, r.top_logprobs, d):
        assert bool(part[[1, 2, 3, 5]].isnan().all()) and not bool(part[[0, 4, 6]].isnan().any())
    assert bool((r.stats[4] == LOW).all()) and not d[4].any()
