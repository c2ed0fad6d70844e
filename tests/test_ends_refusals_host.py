"""Refusals of the operators at a model's two ends that test_ends_host.py does
not make, without a GPU."""
import pytest
import torch

import row_reduction_norm_gb300 as R
from row_reduction_norm_gb300 import _native as N

P = 1 << 20   # a fake, aligned address: never dereferenced, checks fail first


def test_clipping_without_a_largest_norm_is_refused():
    x = torch.ones(4)
    for grads, out in (([x], None), ((x,), [x]), ([], None), ([None], None)):
        with pytest.raises(ValueError, match="max_norm"):
            R.clip_grad_norm(grads, None, out=out)
    with pytest.raises(ValueError, match="max_norm"):
        R.clip_grad_norm([x], max_norm=None)


@pytest.mark.parametrize("stride,dstride", [(100, 101), (128, 100), (100, 200)])
def test_a_gradient_in_place_has_the_logits_stride(stride, dstride):
    for dtype in (N.RMSNORM_F32, N.RMSNORM_BF16):
        assert N.rmsnorm_logprobs_bwd_status(P, 2 * P, 8, 4 * P, 3 * P, None, None, P, 4, 100, stride, dstride, 1.0,
                                             dtype) == N.RMSNORM_EINVAL
