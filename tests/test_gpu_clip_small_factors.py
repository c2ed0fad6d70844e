"""Clipping by factors below fp32's smallest normal number (GB300 only), to the
same bounds as any other: a large norm and a small largest one."""
import pytest
import torch

import ends_ref as ref
from test_gpu_embedding import BF, DEV, F32, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R


@pytest.mark.parametrize("size", [3, 5000, 2000000])
@pytest.mark.parametrize("top,max_norm", [(1e38, 0.1), (3e37, 1e-2), (1e36, 1e-8), (1e30, 2e-10), (1e37, 1e-20), (1e35, 1e-36)])
def test_small_factors(top, max_norm, size):
    g = gen(size)
    max_norm = float(torch.tensor(max_norm))                    # as the call takes it
    for dtype in (BF, F32):
        grads = [normal(g, n, std=0.1).clamp(-1, 1).mul_(top / n ** 0.5 * 3).to(dtype) for n in (size, 7)]
        n = ref.norm(grads)
        assert max_norm / n < 2.0 ** -126 and n < 3.4e38
        want = [ref.clipped(t, n, max_norm) for t in grads]
        out = [torch.empty_like(t) for t in grads]
        got = R.clip_grad_norm(grads, max_norm, out=out)
        assert abs(float(got) - n) <= 8 * ref.U * n
        for o, (y, bound) in zip(out, want):
            ref.assert_within(o, y, bound, "clipped")
        R.clip_grad_norm(grads, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(grads, out))


def test_a_norm_past_fp32s_range():
    """Infinite as fp32 gives it; the tensors are scaled by the norm itself."""
    for size in (64, 1000000):
        grads = [torch.full((size,), 3e38, device=DEV), torch.full((size,), -1.5e38, dtype=BF, device=DEV)]
        n = ref.norm(grads)
        want = [ref.clipped(t, n, 2.0) for t in grads]
        assert n > 3.5e38 and float(R.clip_grad_norm(grads, 2.0)) == float("inf")
        for t, (y, bound) in zip(grads, want):
            ref.assert_within(t, y, bound, "clipped")
