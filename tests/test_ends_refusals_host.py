"""Refusals of the operators at a model's two ends that test_ends_host.py does
not make, without a GPU."""
import pytest
import torch

import row_reduction_norm_gb300 as R


def test_clipping_without_a_largest_norm_is_refused():
    x = torch.ones(4)
    for grads, out in (([x], None), ((x,), [x]), ([], None), ([None], None)):
        with pytest.raises(ValueError, match="max_norm"):
            R.clip_grad_norm(grads, None, out=out)
    with pytest.raises(ValueError, match="max_norm"):
        R.clip_grad_norm([x], max_norm=None)
