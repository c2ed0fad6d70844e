"""Clipping of lists whose tensors have no elements, more of them than a launch
takes (GB300 only): the norm is written all the same."""
import pytest
import torch

from test_gpu_embedding import BF, DEV

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R
    from row_reduction_norm_gb300 import _native as N


@pytest.mark.parametrize("many", [0, 1, 40, 1020, 1021, 1100, 2100])
def test_tensors_without_elements(many):
    a = (N.Grad * max(many, 1))()
    for i in range(many):
        a[i].dtype = i % 2
    need = N.rmsnorm_grad_norm_workspace_bytes()
    room = torch.empty(need, dtype=torch.uint8, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    for call in (lambda n: N.rmsnorm_clip_grads(a, many, 1.0, n.data_ptr(), room.data_ptr(), need, s),
                 lambda n: N.rmsnorm_grad_norm(a, many, n.data_ptr(), room.data_ptr(), need, s)):
        norm = torch.full((3,), 7.0, device=DEV)
        call(norm[1:2])
        assert norm.tolist() == [7.0, 0.0, 7.0]


def test_some_among_many_without_elements():
    none = [torch.empty(0, dtype=BF if i % 2 else torch.float32, device=DEV) for i in range(1050)]
    ones = [torch.full((8,), 0.5, device=DEV), torch.full((32,), 0.25, dtype=BF, device=DEV)]
    for grads in (none + ones, ones + none, none + ones[:1] + none + ones[1:]):
        kept = [t.clone() for t in ones]
        assert float(R.clip_grad_norm(grads, 1.0)) == 2.0
        assert all(torch.equal(t, k / 2) for t, k in zip(ones, kept))
        for t, k in zip(ones, kept):
            t.copy_(k)
