"""The Q+K head norm with rotary positions and its gradient against the
formulas in 64 bits (GB300 only); tolerances in rope_ref.py."""
from fractions import Fraction

import pytest
import torch

import rope_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R
    from row_reduction_norm_gb300 import _native as N

DEV = "cuda"
T = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, device=DEV).normal_(mean, std, generator=g).to(dtype)


def freqs(rot, base=10000.0):
    return (base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)).float().to(DEV)


# (head_dim, rot, sections): halves of 16, 8, 4 and 2 bytes, parts of heads, several axes
SHAPES = [
    (128, 128, (64,)), (64, 64, (8, 12, 12)), (256, 256, (128,)), (512, 512, (256,)), (512, 64, (32,)),
    (80, 80, (8, 16, 16)), (72, 72, (36,)), (96, 48, (24,)), (40, 20, (3, 3, 2, 2)), (80, 20, (10,)), (48, 14, (1, 6)),
    (2, 2, (1,)), (6, 2, (1,)), (500, 250, (125,)), (384, 190, (0, 95)),
]


def inputs(dtype, tokens, q, k, d, rot, sections, seed, norm=True, bias=0.0, extra=1, pos64=True, far=4096):
    g = gen(seed)
    qkv = normal(g, tokens, (q + k + extra) * d, dtype=T[dtype])
    pos = torch.randint(-far, far, (len(sections), tokens), device=DEV, generator=g)
    pos = pos if pos64 else pos.int()
    qw = normal(g, d, dtype=T[dtype], std=0.2, mean=1.0 - bias) if norm else None
    kw = normal(g, d, dtype=T[dtype], std=0.2, mean=1.0 - bias) if norm else None
    return g, qkv, pos, freqs(rot), qw, kw


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,sections", SHAPES)
@pytest.mark.parametrize("tokens,q,k,norm,bias", [(33, 5, 2, True, 0.0), (1, 3, 1, True, 1.0), (70, 2, 0, False, 0.0)])
def test_forward_and_gradient(dtype, interleaved, d, rot, sections, tokens, q, k, norm, bias):
    g, qkv, pos, f, qw, kw = inputs(dtype, tokens, q, k, d, rot, sections, d + rot, norm, bias, pos64=tokens != 33)
    kw_args = dict(q_w=qw, k_w=kw, weight_bias=bias, norm=norm, sections=sections, interleaved=interleaved)
    theta = ref.phases(pos, f, sections)
    keep = qkv.clone()
    y = R.qk_norm_rope(qkv, q, k, d, pos, f, **kw_args)
    want, bound = ref.forward(qkv, q, k, d, theta, rot, interleaved, qw, kw, 1e-6, bias, norm)
    ref.assert_within(y, want, bound, "y")
    assert torch.equal(qkv, keep)

    dy = normal(g, tokens, (q + k) * d, dtype=T[dtype])
    dx, dqw, dkw = R.qk_norm_rope_backward(dy, qkv if norm else None, q, k, d, pos, f, **kw_args)
    want = ref.backward(dy, qkv, q, k, d, theta, rot, interleaved, qw, kw, 1e-6, bias, norm)
    ref.assert_within(dx, want[0], want[1], "dx")
    if norm:
        ref.assert_within(dqw, want[2], want[3], "dq_w")
        ref.assert_within(dkw, want[4], want[5], "dk_w")
    else:
        assert dqw is None and dkw is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tokens_fill_the_device(dtype):
    """Whole-token warps, several tokens a warp in the gradient."""
    tokens, q, k, d = 5003, 8, 2, 64
    g, qkv, pos, f, qw, kw = inputs(dtype, tokens, q, k, d, 64, (32,), 3)
    y = R.qk_norm_rope(qkv, q, k, d, pos, f, q_w=qw, k_w=kw)
    theta = ref.phases(pos, f, (32,))
    want, bound = ref.forward(qkv, q, k, d, theta, 64, False, qw, kw, 1e-6, 0.0, True)
    ref.assert_within(y, want, bound, "y")
    dy = normal(g, tokens, (q + k) * d, dtype=T[dtype])
    out = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, q_w=qw, k_w=kw)
    want = ref.backward(dy, qkv, q, k, d, theta, 64, False, qw, kw, 1e-6, 0.0, True)
    for i, name in enumerate(("dx", "dq_w", "dk_w")):
        ref.assert_within(out[i], want[2 * i], want[2 * i + 1], name)
    again = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, q_w=qw, k_w=kw)
    for a, b in zip(out, again):
        assert torch.equal(a, b), "two runs differ"


def test_a_head_does_not_depend_on_the_batch():
    """One token alone (heads spread over warps) and among others: the same bits."""
    q, k, d = 32, 8, 128
    _, qkv, pos, f, qw, kw = inputs("bf16", 4000, q, k, d, 128, (64,), 5)
    y = R.qk_norm_rope(qkv, q, k, d, pos, f, q_w=qw, k_w=kw)
    for t in (0, 1999, 3999):
        one = R.qk_norm_rope(qkv[t:t + 1], q, k, d, pos[:, t:t + 1].contiguous(), f, q_w=qw, k_w=kw)
        assert torch.equal(one[0], y[t])


@pytest.mark.parametrize("dtype,shift,pad", [("bf16", 0, 0), ("bf16", 4, 8), ("bf16", 2, 6), ("bf16", 1, 3),
                                             ("f32", 1, 5), ("f32", 2, 2)])
def test_strides_offsets_and_in_place(dtype, shift, pad):
    """Views that start off a 16-byte boundary, rows with gaps, in place and
    out of place; what lies around the heads stays as it was."""
    tokens, q, k, d = 19, 4, 2, 64
    g, qkv, pos, f, qw, kw = inputs(dtype, tokens, q, k, d, 64, (32,), 11)
    wide = qkv.shape[1] + pad
    store = normal(g, tokens * wide + shift, dtype=T[dtype])
    view = store[shift:].view(tokens, wide)[:, :qkv.shape[1]]
    view.copy_(qkv)
    keep = store.clone()
    theta = ref.phases(pos, f, (32,))
    want, bound = ref.forward(qkv, q, k, d, theta, 64, False, qw, kw, 1e-6, 0.0, True)
    y = R.qk_norm_rope(view, q, k, d, pos, f, q_w=qw, k_w=kw)
    ref.assert_within(y, want, bound, "strided")
    assert torch.equal(store, keep)
    R.qk_norm_rope(view, q, k, d, pos, f, q_w=qw, k_w=kw, out=view)
    assert torch.equal(view[:, :(q + k) * d], y), "in place"
    view[:, :(q + k) * d] = keep[shift:].view(tokens, wide)[:, :(q + k) * d]
    assert torch.equal(store, keep), "something outside the heads was written"
    # the gradient, into its own gradient's buffer and into a wider one
    dy = normal(g, tokens, (q + k) * d, dtype=T[dtype])
    want = ref.backward(dy, qkv, q, k, d, theta, 64, False, qw, kw, 1e-6, 0.0, True)
    store2 = store.clone()
    dview = store2[shift:].view(tokens, wide)[:, :qkv.shape[1]]
    R.qk_norm_rope_backward(dy, view, q, k, d, pos, f, q_w=qw, k_w=kw, out=dview)
    ref.assert_within(dview[:, :(q + k) * d], want[0], want[1], "dx strided")
    dx = dview[:, :(q + k) * d].clone()
    dview[:, :(q + k) * d] = store[shift:].view(tokens, wide)[:, :(q + k) * d]
    assert torch.equal(store2, store)
    R.qk_norm_rope_backward(dy, view, q, k, d, pos, f, q_w=qw, k_w=kw, out=dy)
    ref.assert_within(dy, want[0], want[1], "dx in place")
    assert dx.shape == dy.shape


def test_far_positions_lose_nothing():
    """Positions up to 2^40 of either sign: pairs (1, 0) come out as the
    cosine and sine of the exact product, taken modulo 2 pi with rationals."""
    f = torch.tensor([1.0, 0.5, 0.1, 3.14159265, 1e-3, 1e-7, 2.5e-39, 0.0, 7.0, -0.25], device=DEV)
    pos = torch.tensor([[0, 1, -1, 7, 4097, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), (1 << 40) + 12345]],
                       device=DEV)
    d = 2 * len(f)
    x = torch.zeros(pos.shape[1], d, device=DEV)
    x[:, :len(f)] = 1.0
    y = R.qk_norm_rope(x, 1, 0, d, pos, f, norm=False).cpu().double()
    two_pi = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)
    for t, p in enumerate(pos[0].tolist()):
        for i, v in enumerate(f.tolist()):
            turns = Fraction(p) * Fraction(v) / two_pi
            angle = torch.tensor(float((turns - round(turns)) * two_pi), dtype=torch.float64)
            # fp32 sine and cosine 3e-7; the step of a position is M K 2^s, K = 2^64 / 2 pi off by at
            # most 1/2 and M 2^s = |v|, so the product is off by |v| / 2, the shift drops less than 1 more:
            # under 1 + |v| units of 2^-64 turns, 2 pi (1 + |v|) 2^-64 of angle, for each of |p| steps
            slack = 3e-7 + 6.2832 * (1 + abs(v)) * abs(p) * 2.0 ** -64
            assert abs(float(y[t, i] - torch.cos(angle))) <= slack, (p, v)
            assert abs(float(y[t, len(f) + i] - torch.sin(angle))) <= slack, (p, v)


def test_infinities_and_nan_stay_in_their_head():
    """A NaN or infinity makes its own head NaN where the formula does, and
    only what is not turned passes through."""
    q, k, d, rot = 2, 1, 64, 32
    _, qkv, pos, f, _, _ = inputs("f32", 4, q, k, d, rot, (16,), 2, norm=False)
    qkv[1, 3] = float("nan")
    qkv[2, d + 40] = float("inf")       # past rot: not turned
    y = R.qk_norm_rope(qkv, q, k, d, pos, f, norm=False)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 3] = want[1, 3 + 16] = want[2, d + 40] = True
    assert torch.equal(bad, want) and y[2, d + 40] == float("inf")
    # with the norm the whole head is lost, its neighbours are not
    w = torch.ones(d, device=DEV)
    y = R.qk_norm_rope(qkv, q, k, d, pos, f, q_w=w, k_w=w)
    rows = torch.isnan(y.view(4, q + k, d)).any(-1)
    assert rows.nonzero().tolist() == [[1, 0], [2, 1]]


def test_zero_rows_and_eps():
    """A row of zeros: y = 0 with eps > 0; the gradient of the weights takes
    nothing from heads that are not there, with eps = 0 too."""
    q, k, d = 3, 2, 64      # 3 and 2 heads in groups of 8: idle heads in every warp
    g, qkv, pos, f, qw, kw = inputs("f32", 9, q, k, d, 64, (32,), 4)
    dy = normal(g, 9, (q + k) * d, dtype=torch.float32)
    theta = ref.phases(pos, f, (32,))
    out = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, q_w=qw, k_w=kw, eps=0.0)
    want = ref.backward(dy, qkv, q, k, d, theta, 64, False, qw, kw, 0.0, 0.0, True)
    for i in range(3):
        ref.assert_within(out[i], want[2 * i], want[2 * i + 1], ("dx", "dq_w", "dk_w")[i])
    qkv[4] = 0.0
    y = R.qk_norm_rope(qkv, q, k, d, pos, f, q_w=qw, k_w=kw)
    assert bool((y[4] == 0).all())


def test_no_tokens():
    d = 64
    f, w = freqs(64), torch.ones(d, device=DEV)
    x = torch.empty(0, 3 * d, device=DEV)
    pos = torch.empty(0, device=DEV, dtype=torch.int64)
    assert R.qk_norm_rope(x, 2, 1, d, pos, f, q_w=w, k_w=w).shape == (0, 3 * d)
    dx, dq, dk = R.qk_norm_rope_backward(x, x, 2, 1, d, pos, f, q_w=w, k_w=w)
    assert dx.shape == (0, 3 * d) and bool((dq == 0).all()) and bool((dk == 0).all())


def test_heads_without_queries_or_keys():
    d = 64
    g, qkv, pos, f, qw, kw = inputs("f32", 21, 0, 3, d, 64, (32,), 6)
    dy = normal(g, 21, 3 * d, dtype=torch.float32)
    dx, dq, dk = R.qk_norm_rope_backward(dy, qkv, 0, 3, d, pos, f, q_w=qw, k_w=kw)
    want = ref.backward(dy, qkv, 0, 3, d, ref.phases(pos, f, (32,)), 64, False, qw, kw, 1e-6, 0.0, True)
    ref.assert_within(dx, want[0], want[1], "dx")
    ref.assert_within(dk, want[4], want[5], "dk_w")
    assert bool((dq == 0).all())


def test_gradient_against_differences():
    """Central differences of the forward in 64 bits, along random directions."""
    tokens, q, k, d, sections = 6, 2, 1, 16, (3, 5)
    g, qkv, pos, f, qw, kw = inputs("f32", tokens, q, k, d, 16, sections, 9, far=50)
    theta = ref.phases(pos, f, sections)
    dy = normal(g, tokens, (q + k) * d, dtype=torch.float32)
    dx, dq, dk = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, q_w=qw, k_w=kw, sections=sections)

    def loss(x, a, b):
        y, _ = ref.forward(x, q, k, d, theta, 16, False, a, b, 1e-6, 0.0, True)
        return float((y.reshape(tokens, -1) * dy.double()).sum())

    h = 1e-5
    for seed in range(4):
        gg = gen(100 + seed)
        vx = normal(gg, tokens, (q + k) * d, dtype=torch.float64)
        va, vb = normal(gg, d, dtype=torch.float64), normal(gg, d, dtype=torch.float64)
        x, a, b = qkv[:, :(q + k) * d].double(), qw.double(), kw.double()
        # float64 tensors: half_step of the reference's bound is that type's, unused here
        num = (loss(x + h * vx, a + h * va, b + h * vb) - loss(x - h * vx, a - h * va, b - h * vb)) / (2 * h)
        parts = [(dx.double() * vx), (dq.double() * va), (dk.double() * vb)]
        ana = float(sum(p.sum() for p in parts))
        size = float(sum(p.abs().sum() for p in parts))
        assert abs(num - ana) <= 1e-5 * size, (num, ana)


def test_streams_threads_and_graphs():
    """On a side stream, captured into two graphs that share a workspace and
    replayed with new inputs, and from two host threads at once."""
    import threading
    tokens, q, k, d = 300, 8, 2, 128
    g, qkv, pos, f, qw, kw = inputs("bf16", tokens, q, k, d, 128, (64,), 21)
    dy = normal(g, tokens, (q + k) * d, dtype=torch.bfloat16)
    args = dict(q_w=qw, k_w=kw)
    y0 = R.qk_norm_rope(qkv, q, k, d, pos, f, **args)
    d0 = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, **args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y1 = R.qk_norm_rope(qkv, q, k, d, pos, f, stream=s, **args)
    d1 = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, stream=s, **args)
    s.synchronize()
    assert torch.equal(y0, y1) and all(torch.equal(a, b) for a, b in zip(d0, d1))

    ws = torch.empty(R.rmsnorm_qk_rope_bwd_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append((R.qk_norm_rope(qkv, q, k, d, pos, f, **args),
                         R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, workspace=ws, **args)))
        graphs.append(gr)
    qkv.copy_(normal(g, *qkv.shape, dtype=qkv.dtype))
    pos.add_(17)
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    y2 = R.qk_norm_rope(qkv, q, k, d, pos, f, **args)
    d2 = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, **args)
    for y, dd in outs:
        assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(dd, d2))

    errors = []

    def work():
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                got = [R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, **args) for _ in range(10)]
            st.synchronize()
            for one in got:
                assert all(torch.equal(a, b) for a, b in zip(one, d2))
        except Exception as e:   # reported below
            errors.append(repr(e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_python_refusals():
    d = 64
    _, qkv, pos, f, qw, kw = inputs("bf16", 4, 2, 1, d, 64, (32,), 1)
    for bad in (dict(sections=(31,)), dict(sections=(8, 8, 8, 4, 4)), dict(q_w=qw), dict(q_w=qw[:32], k_w=kw),
                dict(q_w=qw.float(), k_w=kw), dict(out=torch.empty(3, 3 * d, device=DEV, dtype=qkv.dtype)),
                dict(out=torch.empty(4, 2 * d, device=DEV, dtype=qkv.dtype)), dict(norm=False, q_w=qw, k_w=kw)):
        with pytest.raises((ValueError, N.RmsNormError)):
            R.qk_norm_rope(qkv, 2, 1, d, pos, f, **bad)
    with pytest.raises(ValueError):
        R.qk_norm_rope(qkv, 2, 1, d, pos[:, :3], f)
    with pytest.raises(ValueError):
        R.qk_norm_rope(qkv, 2, 1, d, pos.float(), f)
    with pytest.raises(ValueError):
        R.qk_norm_rope(qkv, 2, 1, d, pos, f.double())
    with pytest.raises(ValueError):
        R.qk_norm_rope(qkv, 4, 1, d, pos, f)
    with pytest.raises(ValueError):
        R.qk_norm_rope_backward(qkv, None, 2, 1, d, pos, f, q_w=qw, k_w=kw)
    with pytest.raises(ValueError):
        R.qk_norm_rope_backward(qkv, qkv, 2, 1, d, pos, f, q_w=qw, k_w=kw,
                                workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(N.RmsNormError):      # a broadcast gradient has no row stride
        R.qk_norm_rope_backward(qkv[:1].expand(4, -1), qkv, 2, 1, d, pos, f, q_w=qw, k_w=kw)
