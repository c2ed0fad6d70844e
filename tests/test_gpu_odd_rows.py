"""Rows of odd widths in the dropout and gradient operators (GB300 only): the
narrowest ones, several to a 16-byte chunk, and equal bits in every batch;
tolerances in drop_ref.py."""
import pytest
import torch

import drop_ref as ref
from rope_ref import assert_within
from test_gpu_rope import DEV, T, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R

SEED, OFFSET = 0xABCDEF, 41


# rows that end in the middle of the chunk their tensor ends in, and on its end
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hidden", range(1, 18))
def test_rows_narrower_than_a_chunk(dtype, hidden):
    t, p = T[dtype], 0.25
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device=DEV)
    for rows in (5, 4096, 4097, 4098, 4099, 4101, 4103, 4110):
        g = gen(hidden + rows)
        x, res, dy, dh = (normal(g, rows, hidden, dtype=t) for _ in range(4))
        w = normal(g, hidden, dtype=t, std=0.2, mean=1.0)
        keep = ref.kept(rows, hidden, p, SEED, OFFSET)
        y, h = R.rms_norm_dropout(x, res, p, rng, w)
        assert torch.equal(h.cpu(), ref.forward_h(x, res, keep, p)), rows
        assert_within(y, *ref.norm(h, w, 1e-6, 0.0), f"y, {rows} rows")
        want = ref.backward(dy, h, w, dh, keep.to(DEV), p, 1e-6, 0.0)
        got = R.rms_norm_dropout_backward(dy, h, p, rng, w, dh)
        for i, name in enumerate(("dresidual", "dx", "dw")):
            assert_within(got[i], want[2 * i], want[2 * i + 1], f"{name}, {rows} rows")


# widths on both sides of every border between the kernels' shapes; the row
# counts are on both sides of those from which another kernel takes the rows
ODD = {"bf16": (7, 13, 64, 101, 241, 249, 250, 251, 501, 511, 513, 1001, 1017, 1018, 1021, 1535, 1536, 2041, 2042, 2047, 2999, 4095,
                8191, 12001),
       "f32": (3, 5, 100, 101, 125, 126, 127, 253, 254, 501, 509, 510, 511, 513, 1001, 1021, 1022, 1023, 2044, 2045, 2046, 2047,
               3001, 4093, 6001, 8187)}


@pytest.mark.parametrize("dtype,hidden", [(d, h) for d in ODD for h in ODD[d]])
def test_a_row_has_the_same_bits_in_every_batch(dtype, hidden):
    """y and the gradients of a row's input, whatever the number of rows and the row's place among them."""
    t, g = T[dtype], gen(hidden)
    rows = 5000 if hidden < 900 else 4600
    x, res, dy, dh = (normal(g, rows, hidden, dtype=t) for _ in range(4))
    w = normal(g, hidden + 1, dtype=t, std=0.2, mean=1.0)[1:]   # off the boundary
    y, h = R.rms_norm_dropout(x, res, 0.0, None, w, weight_bias=0.5)
    dx, _ = R.rms_norm_backward(dy, h, w, dh, weight_bias=0.5)
    bare, _ = R.rms_norm_backward(dy, h)
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device=DEV)
    dres, _, _ = R.rms_norm_dropout_backward(dy, h, 0.25, rng, w, dh, weight_bias=0.5)
    assert torch.equal(dres, dx)
    for first, n in ((0, 4095), (0, 4096), (1, 4097), (5, 1100), (3, 300), (rows - 9, 9), (rows - 2, 1), (17, 1), (22, 2)):
        cut = lambda v: v[first:first + n].clone()
        y2, h2 = R.rms_norm_dropout(cut(x), cut(res), 0.0, None, w, weight_bias=0.5)
        assert torch.equal(h2, cut(h)) and torch.equal(y2, cut(y)), (first, n)
        d2, _ = R.rms_norm_backward(cut(dy), cut(h), w, cut(dh), weight_bias=0.5)
        assert torch.equal(d2, cut(dx)), (first, n)
        assert torch.equal(R.rms_norm_backward(cut(dy), cut(h))[0], cut(bare)), (first, n)
