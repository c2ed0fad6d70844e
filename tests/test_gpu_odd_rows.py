"""Rows of odd widths in the dropout and gradient operators (GB300 only): the
narrowest ones, several to a 16-byte chunk; tolerances in drop_ref.py."""
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
