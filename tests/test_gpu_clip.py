"""The norm of many tensors and their clipping (GB300 only) against the formula
in 64 bits, with the bounds of ends_ref.py."""
import pytest
import torch

import ends_ref as ref
from test_gpu_embedding import BF, DEV, F32, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R


def check(grads, ratio, in_place=False):
    n = ref.norm(grads)
    want = [ref.clipped(g, n, ratio * n) for g in grads]
    assert abs(float(R.grad_norm(grads)) - n) <= 8 * ref.U * n
    if in_place:
        out = [g.clone() for g in grads]
        got = R.clip_grad_norm(out, ratio * n)
    else:
        kept = [g.clone() for g in grads]
        out = [torch.empty_like(g) for g in grads]
        got = R.clip_grad_norm(grads, ratio * n, out=out)
        assert all(torch.equal(a, b) for a, b in zip(kept, grads))
    assert got.shape == (1,) and got.dtype is F32 and abs(float(got) - n) <= 8 * ref.U * n
    for o, (y, bound) in zip(out, want):
        ref.assert_within(o, y, bound, "clipped")
    if ratio > 1:
        assert all(torch.equal(o, g) for o, g in zip(out, grads))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ratio", [0.1, 0.77, 2.0])
@pytest.mark.parametrize("sizes", [[1], [7, 1, 0, 9], [1000] * 39, [33] * 40, [5] * 41, [100] * 1020, [65] * 1021, [3] * 2500,
                                   [16384, 16385, 1, 2048, 300001], [5000000, 17, 8192]])
def test_lists_of_tensors(sizes, ratio, in_place):
    g = gen(len(sizes))
    check([normal(g, n, dtype=BF if i % 3 else F32, std=0.02) for i, n in enumerate(sizes)], ratio, in_place)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off,ooff", [(0, 1), (1, 1), (3, 0), (7, 7), (2, 6), (5, 4)])
def test_unaligned_tensors_and_their_neighbours(off, ooff, dtype):
    g = gen(off)
    for n in (1, 6, 9, 100, 16384, 40001):
        room = normal(g, n + off + 9, dtype=dtype)
        grad = room[off:off + n]
        to = torch.full((n + ooff + 16,), 7.0, dtype=dtype, device=DEV)
        norm = ref.norm([grad])
        R.clip_grad_norm([grad], 0.5 * norm, out=[to[ooff:ooff + n]])
        ref.assert_within(to[ooff:ooff + n], *ref.clipped(grad, norm, 0.5 * norm), "unaligned")
        assert bool((to[:ooff] == 7.0).all()) and bool((to[ooff + n:] == 7.0).all())
        kept = room.clone()
        R.clip_grad_norm([grad], 0.5 * norm)
        assert torch.equal(room[:off], kept[:off]) and torch.equal(room[off + n:], kept[off + n:])
        assert torch.equal(grad, to[ooff:ooff + n])


@pytest.mark.parametrize("size", [3, 4097, 3000000])
def test_values_whose_squares_fp32_cannot_hold(size):
    g = gen(size)
    for std in (1e25, 1e37, 1e-25, 1e-37):
        for dtype in (BF, F32):
            grads = [normal(g, size, dtype=F32).mul_(std).to(dtype), normal(g, 5).mul_(std)]
            n = ref.norm(grads)
            if n > 3e38:
                continue
            # a subnormal element is a value like others; the norm itself is rounded to fp32
            assert abs(float(R.grad_norm(grads)) - n) <= 8 * ref.U * n + 2.0 ** -149
    ones = [torch.full((size,), 1e-30, device=DEV), torch.full((100,), 1e19, device=DEV)]
    assert abs(float(R.grad_norm(ones)) - 1e20) <= 8 * ref.U * 1e20


def test_nothing_zeros_infinities_and_nan():
    zero = [torch.zeros(5000, device=DEV), torch.zeros(3, dtype=BF, device=DEV)]
    assert float(R.clip_grad_norm(zero, 1.0)) == 0.0 and not zero[0].any()
    assert float(R.grad_norm([torch.empty(0, device=DEV)])) == 0.0
    assert float(R.clip_grad_norm([None, torch.empty(0, device=DEV)], 1.0)) == 0.0
    for dtype in (BF, F32):
        a = [torch.ones(100, dtype=dtype, device=DEV), torch.ones(7, device=DEV)]
        a[0][3] = float("inf")
        assert float(R.clip_grad_norm(a, 1.0)) == float("inf")
        assert bool(a[0][3].isnan()) and not a[0][4:].any() and not a[1].any()
        b = [torch.ones(100, dtype=dtype, device=DEV), torch.ones(7, device=DEV)]
        b[0][99] = float("nan")
        assert bool(R.clip_grad_norm(b, 1.0).isnan().all()) and bool(b[0].isnan().all()) and bool(b[1].isnan().all())
    c = [torch.ones(4, device=DEV)]
    assert float(R.clip_grad_norm(c, float("inf"))) == 2.0 and bool((c[0] == 1).all())
    assert float(R.clip_grad_norm(c, 0.0)) == 2.0 and not c[0].any()


def test_none_entries_and_shapes():
    g = gen(3)
    grads = [normal(g, 4, 5), None, normal(g, 3, 2, 2, dtype=BF), None]
    kept = [x.clone() for x in grads if x is not None]
    n = ref.norm(kept)
    assert abs(float(R.clip_grad_norm(tuple(grads), 0.5 * n)) - n) <= 8 * ref.U * n
    for x, k in zip([x for x in grads if x is not None], kept):
        ref.assert_within(x, *ref.clipped(k, n, 0.5 * n), "in a list with Nones")


def test_a_tensor_past_32_bit_offsets():
    n = 2 ** 31 + 2 ** 20 + 3                                    # 4.3 GB
    x = torch.zeros(n, dtype=BF, device=DEV)
    at = torch.tensor([0, 2 ** 30, 2 ** 31 - 1, 2 ** 31, n - 1], device=DEV)
    x[at] = 2.0
    assert abs(float(R.clip_grad_norm([x], 1.0)) - 20 ** 0.5) <= 8 * ref.U * 20 ** 0.5
    assert bool(((x[at].float() * 20 ** 0.5 - 2).abs() < 0.02).all()) and int((x != 0).sum()) == 5


def test_the_same_bits_every_time():
    g = gen(6)
    grads = [normal(g, 1 + 7919 * i, dtype=BF if i % 2 else F32) for i in range(60)]
    first = R.grad_norm(grads)
    for _ in range(4):
        assert torch.equal(first, R.grad_norm(grads))


def test_refusals_of_python_calls():
    x = torch.ones(4, 6, device=DEV)
    bad = [lambda: R.clip_grad_norm([x.t()], 1.0), lambda: R.clip_grad_norm([x, x.cpu()], 1.0),
           lambda: R.clip_grad_norm([x], 1.0, out=[x[:3]]), lambda: R.clip_grad_norm([x], 1.0, out=[x.to(BF)]),
           lambda: R.clip_grad_norm([x], 1.0, out=[None]),
           lambda: R.grad_norm([x], workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        R.grad_norm([x.half()])
    for m in (-1.0, float("nan")):
        with pytest.raises(R.RmsNormError):
            R.clip_grad_norm([x], m)
    assert bool((x == 1).all())
