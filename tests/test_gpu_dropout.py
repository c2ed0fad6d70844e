"""Residual dropout with RMSNorm and the gradients, against the formulas in 64
bits (GB300 only); tolerances in drop_ref.py."""
import pytest
import torch

import drop_ref as ref
from rope_ref import assert_within
from test_gpu_rope import DEV, T, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R
    from row_reduction_norm_gb300 import _native as N

SEED, OFFSET = 0x1234567_89ABCDEF, (1 << 40) + 3


def rng_of(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


# (rows, hidden): every kernel shape and the borders between them
SHAPES = [(1, 1), (3, 7), (5, 64), (40, 64), (33, 100), (9, 264), (7, 576), (64, 1000), (300, 1001), (20, 2048),
          (4, 4096), (5, 4097), (3, 8192), (3, 12288), (2, 16384), (2, 16392), (2, 20480), (2, 32768), (2, 40000),
          (3, 49153), (2, 65535), (1, 65536)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("p,weight,bias,with_dh", [(0.1, True, 0.0, True), (0.5, False, 0.0, False), (0.0, True, 1.0, True),
                                                   (0.25, True, 0.0, False)])
def test_forward_and_gradient(dtype, rows, hidden, p, weight, bias, with_dh):
    g = gen(rows * 7 + hidden)
    t = T[dtype]
    x, res = normal(g, rows, hidden, dtype=t), normal(g, rows, hidden, dtype=t)
    w = normal(g, hidden, dtype=t, std=0.2, mean=1.0 - bias) if weight else None
    rng = rng_of() if p else None
    y, h = R.rms_norm_dropout(x, res, p, rng, w=w, weight_bias=bias)
    keep = ref.kept(rows, hidden, p, SEED, OFFSET)
    assert torch.equal(h.cpu(), ref.forward_h(x, res, keep, p)), "residual_out"
    want, bound = ref.norm(h, w, 1e-6, bias)
    assert_within(y, want, bound, "y")

    dy = normal(g, rows, hidden, dtype=t)
    dh = normal(g, rows, hidden, dtype=t) if with_dh else None
    keep = keep.to(DEV)
    want = ref.backward(dy, h, w, dh, keep, p, 1e-6, bias)
    dres, dx, dw = R.rms_norm_dropout_backward(dy, h, p, rng, w=w, dresidual_out=dh, weight_bias=bias)
    assert_within(dres, want[0], want[1], "dresidual")
    assert_within(dx, want[2], want[3], "dx")
    if weight:
        assert_within(dw, want[4], want[5], "dw")
    else:
        assert dw is None
    only, dw2 = R.rms_norm_backward(dy, h, w=w, dresidual_out=dh, weight_bias=bias)
    assert torch.equal(only, dres) and (dw2 is None or torch.equal(dw2, dw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden", [(5000, 64), (3001, 576), (2003, 1001), (1000, 4096), (700, 8192), (400, 16384),
                                         (310, 20480)])
def test_many_rows_a_block(dtype, rows, hidden):
    g = gen(hidden)
    t = T[dtype]
    x, res, w = normal(g, rows, hidden, dtype=t), normal(g, rows, hidden, dtype=t), normal(g, hidden, dtype=t)
    rng = rng_of()
    keep = ref.kept(rows, hidden, 0.1, SEED, OFFSET)
    y, h = R.rms_norm_dropout(x, res, 0.1, rng, w=w)
    assert torch.equal(h.cpu(), ref.forward_h(x, res, keep, 0.1))
    want, bound = ref.norm(h, w, 1e-6, 0.0)
    assert_within(y, want, bound, "y")
    dy, dh = normal(g, rows, hidden, dtype=t), normal(g, rows, hidden, dtype=t)
    want = ref.backward(dy, h, w, dh, keep.to(DEV), 0.1, 1e-6, 0.0)
    out = R.rms_norm_dropout_backward(dy, h, 0.1, rng, w=w, dresidual_out=dh)
    for i, name in enumerate(("dresidual", "dx", "dw")):
        assert_within(out[i], want[2 * i], want[2 * i + 1], name)
    again = R.rms_norm_dropout_backward(dy, h, 0.1, rng, w=w, dresidual_out=dh)
    assert all(torch.equal(a, b) for a, b in zip(out, again)), "two runs differ"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hidden", [576, 1001, 2048, 8191, 20480])
def test_unaligned_tensors_and_in_place(dtype, hidden):
    """Tensors one element off a 16-byte boundary (same values up to rounding,
    the same mask), and every allowed use of an input's buffer as an output."""
    rows, t, rng = 6, T[dtype], rng_of()
    g = gen(5)
    x, res, w = normal(g, rows, hidden, dtype=t), normal(g, rows, hidden, dtype=t), normal(g, hidden, dtype=t)
    dy, dh = normal(g, rows, hidden, dtype=t), normal(g, rows, hidden, dtype=t)
    y, h = R.rms_norm_dropout(x, res, 0.1, rng, w=w)
    dres, dx, dw = R.rms_norm_dropout_backward(dy, h, 0.1, rng, w=w, dresidual_out=dh)
    store = torch.full((rows * hidden + 2,), 3.0, dtype=t, device=DEV)

    def off(v):
        s = store.clone()
        o = s[1:-1].view(rows, hidden)
        o.copy_(v)
        return s, o

    xs, xo = off(x)
    hs, ho = off(torch.zeros_like(x))
    y2, h2 = R.rms_norm_dropout(xo, res, 0.1, rng, w=w, residual_out=ho)
    assert torch.equal(h2, h)
    want, bound = ref.norm(h, w, 1e-6, 0.0)
    assert_within(y2, want, bound, "y, unaligned")
    assert float(hs[0]) == 3.0 and float(hs[-1]) == 3.0 and float(xs[-1]) == 3.0
    keep = ref.kept(rows, hidden, 0.1, SEED, OFFSET).to(DEV)
    want = ref.backward(dy, h, w, dh, keep, 0.1, 1e-6, 0.0)
    _, dyo = off(dy)
    ds, do = off(torch.zeros_like(x))
    out = R.rms_norm_dropout_backward(dyo, h, 0.1, rng, w=w, dresidual_out=dh, dresidual=do)
    for i, name in enumerate(("dresidual", "dx", "dw")):
        assert_within(out[i], want[2 * i], want[2 * i + 1], name + ", unaligned")
    assert float(ds[0]) == 3.0 and float(ds[-1]) == 3.0

    for a, b in (("x", "res"), ("res", "x")):      # y over one input, residual_out over the other
        c = {"x": x.clone(), "res": res.clone()}
        y3, h3 = R.rms_norm_dropout(c["x"], c["res"], 0.1, rng, w=w, out=c[a], residual_out=c[b])
        assert torch.equal(y3, y) and torch.equal(h3, h)
    for a, b in (("dy", "h"), ("h", "dh"), ("dh", "dy")):
        c = {"dy": dy.clone(), "h": h.clone(), "dh": dh.clone()}
        o = R.rms_norm_dropout_backward(c["dy"], c["h"], 0.1, rng, w=w, dresidual_out=c["dh"], dresidual=c[a], dx=c[b])
        assert torch.equal(o[0], dres) and torch.equal(o[1], dx) and torch.equal(o[2], dw), (a, b)


def test_a_row_does_not_depend_on_the_batch_but_on_its_place():
    g = gen(3)
    x, res, w = (normal(g, 600, 2048, dtype=torch.bfloat16) for _ in range(3))
    y, h = R.rms_norm_dropout(x, res, 0.1, rng_of(), w=w[0])
    y2, h2 = R.rms_norm_dropout(x[:5], res[:5], 0.1, rng_of(), w=w[0])
    assert torch.equal(y[:5], y2) and torch.equal(h[:5], h2)


def test_dropped_places_add_nothing():
    """NaN and infinity in x where it is dropped leave no trace; an infinite
    row loses itself only."""
    rows, hidden = 8, 512
    g = gen(9)
    x, res = normal(g, rows, hidden, dtype=torch.float32), normal(g, rows, hidden, dtype=torch.float32)
    keep = ref.kept(rows, hidden, 0.5, SEED, OFFSET).to(DEV)
    bad = torch.where(keep, x, torch.full_like(x, float("nan")))
    y, h = R.rms_norm_dropout(x, res, 0.5, rng_of())
    y2, h2 = R.rms_norm_dropout(bad, res, 0.5, rng_of())
    assert torch.equal(y, y2) and torch.equal(h, h2)
    res[3, 100] = float("inf")
    y3, h3 = R.rms_norm_dropout(x, res, 0.5, rng_of())
    assert torch.equal(torch.isnan(y3).any(-1).nonzero().flatten(), torch.tensor([3], device=DEV))
    ok = [i for i in range(rows) if i != 3]
    assert torch.equal(y3[ok], y[ok])


def test_idle_row_slots_add_nothing_without_eps():
    """33 rows in groups of 8: the empty slots of the last group must not reach
    dw, with eps = 0 too."""
    g = gen(4)
    dy, h, w = normal(g, 33, 576, dtype=torch.float32), normal(g, 33, 576, dtype=torch.float32), normal(g, 576,
                                                                                                    dtype=torch.float32)
    want = ref.backward(dy, h, w, None, None, 0.0, 0.0, 0.0)
    dx, dw = R.rms_norm_backward(dy, h, w=w, eps=0.0)
    assert_within(dx, want[0], want[1], "dx")
    assert_within(dw, want[4], want[5], "dw")


def test_no_rows():
    x = torch.empty(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    y, h = R.rms_norm_dropout(x, x, 0.1, rng_of(), w=w)
    assert y.shape == (0, 64) and h.shape == (0, 64)
    dx, dw = R.rms_norm_backward(x, x, w=w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_gradient_against_differences():
    """Central differences of the formulas in 64 bits, with the mask held."""
    rows, hidden, p, eps = 5, 48, 0.25, 1e-5
    g = gen(11)
    x, res, w = (normal(g, rows, hidden, dtype=torch.float32) for _ in range(3))
    w = w[0].contiguous()
    keep = ref.kept(rows, hidden, p, SEED, OFFSET).to(DEV)
    s = 65536.0 / (65536 - ref.threshold(p))
    dy, dh = normal(g, rows, hidden, dtype=torch.float32), normal(g, rows, hidden, dtype=torch.float32)
    y, h = R.rms_norm_dropout(x, res, p, rng_of(), w=w, eps=eps)
    dres, dx, dw = R.rms_norm_dropout_backward(dy, h, p, rng_of(), w=w, dresidual_out=dh, eps=eps)

    def loss(a, b, c):
        f = b + torch.where(keep, a * s, torch.zeros_like(a))
        n = f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps) * c
        return float((n * dy.double()).sum() + (f * dh.double()).sum())

    step = 1e-5
    for seed in range(4):
        gg = gen(50 + seed)
        va, vb = normal(gg, rows, hidden, dtype=torch.float64), normal(gg, rows, hidden, dtype=torch.float64)
        vc = normal(gg, hidden, dtype=torch.float64)
        a, b, c = x.double(), res.double(), w.double()
        num = (loss(a + step * va, b + step * vb, c + step * vc) - loss(a - step * va, b - step * vb, c - step * vc)) / (
            2 * step)
        parts = [dx.double() * va, dres.double() * vb, dw.double() * vc]
        size = float(sum(q.abs().sum() for q in parts))
        assert abs(num - float(sum(q.sum() for q in parts))) <= 1e-5 * size


def test_streams_graphs_and_new_masks():
    """On a side stream; captured once and replayed with the offset advanced
    on the device: another mask each time, the same in both directions."""
    rows, hidden, p = 200, 2048, 0.1
    g = gen(6)
    x, res, dy = (normal(g, rows, hidden, dtype=torch.bfloat16) for _ in range(3))
    w = normal(g, hidden, dtype=torch.bfloat16)
    rng = rng_of(5, 0)
    y0, h0 = R.rms_norm_dropout(x, res, p, rng, w=w)
    d0 = R.rms_norm_dropout_backward(dy, h0, p, rng, w=w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y1, h1 = R.rms_norm_dropout(x, res, p, rng, w=w, stream=s)
    d1 = R.rms_norm_dropout_backward(dy, h1, p, rng, w=w, stream=s)
    s.synchronize()
    assert torch.equal(y0, y1) and torch.equal(h0, h1) and all(torch.equal(a, b) for a, b in zip(d0, d1))
    ws = torch.empty(R.rmsnorm_bwd_workspace_bytes(rows, hidden, N.RMSNORM_BF16), dtype=torch.uint8, device=DEV)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y, h = R.rms_norm_dropout(x, res, p, rng, w=w)
            d = R.rms_norm_dropout_backward(dy, h, p, rng, w=w, workspace=ws)
        graphs.append((gr, y, h, d))
    seen = []
    for offset in (0, 1, 2):
        rng[1] = offset
        for gr, *_ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        keep = ref.kept(rows, hidden, p, 5, offset)
        for _, y, h, d in graphs:
            assert torch.equal(h.cpu(), ref.forward_h(x, res, keep, p))
            want = ref.backward(dy, h, w, None, keep.to(DEV), p, 1e-6, 0.0)
            for i in range(3):
                assert_within(d[i], want[2 * i], want[2 * i + 1], ("dresidual", "dx", "dw")[i])
        seen.append(graphs[0][2].clone())
    assert torch.equal(seen[0], h0) and not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_python_refusals():
    x = torch.zeros(4, 64, device=DEV)
    w, rng = torch.ones(64, device=DEV), rng_of()
    for call in (lambda: R.rms_norm_dropout(x, x[:2], 0.1, rng), lambda: R.rms_norm_dropout(x, x, 0.1, None),
                 lambda: R.rms_norm_dropout(x, x, 0.1, rng.cpu()), lambda: R.rms_norm_dropout(x, x, 0.1, rng.int()),
                 lambda: R.rms_norm_dropout(x, x, 0.1, rng[:1]), lambda: R.rms_norm_dropout(x, x, 1.0, rng),
                 lambda: R.rms_norm_dropout(x, x, 0.1, rng, w=w[:32]),
                 lambda: R.rms_norm_dropout(x, x, 0.1, rng, weight_bias=1.0),
                 lambda: R.rms_norm_dropout(x.t(), x.t(), 0.1, rng),
                 lambda: R.rms_norm_dropout(x, x, 0.1, rng, out=x, residual_out=x),
                 lambda: R.rms_norm_backward(x, x.bfloat16()), lambda: R.rms_norm_backward(x, x, dresidual_out=x[0]),
                 lambda: R.rms_norm_backward(x, x, w=w, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
                 lambda: R.rms_norm_dropout_backward(x, x, 0.1, rng, dresidual=x, dx=x)):
        with pytest.raises((ValueError, N.RmsNormError)):
            call()


# widths that are no multiple of 16 bytes: each number of chunks a thread takes, and rows a block
@pytest.mark.parametrize("dtype,hidden", [
    ("bf16", 7), ("bf16", 13), ("bf16", 241), ("bf16", 505), ("bf16", 1001), ("bf16", 2047), ("bf16", 2999),
    ("bf16", 4090), ("bf16", 6001), ("bf16", 8191), ("bf16", 12001), ("bf16", 16377), ("bf16", 16379),
    ("f32", 5), ("f32", 121), ("f32", 253), ("f32", 1001), ("f32", 1531), ("f32", 2045), ("f32", 3001), ("f32", 4093),
    ("f32", 6002), ("f32", 8189), ("f32", 8191),
])
@pytest.mark.parametrize("few", [True, False])
def test_widths_off_the_boundary(dtype, hidden, few):
    """Rows that start anywhere between two boundaries; infinities in the rows
    beside a finite one stay out of it, and what is behind the tensors is left alone."""
    rows = 11 if few else 20000 if hidden < 300 else 4501 if hidden < 2100 else 701
    t, p, g = T[dtype], 0.25, gen(hidden + rows)

    def within(fill=None):   # a tensor of rows, on a boundary, with something else behind it
        room = torch.full((rows * hidden + 64,), 7.5, dtype=t, device=DEV)
        v = room[:rows * hidden].view(rows, hidden)
        if fill is not None:
            v.copy_(fill)
        return room, v

    src = [normal(g, rows, hidden, dtype=t) for _ in range(4)]
    src[1][4] = float("inf")
    (_, x), (_, res), (_, dy), (_, dh) = (within(v) for v in src)
    w = normal(g, hidden + 1, dtype=t, std=0.2, mean=1.0)[1:]
    rng = rng_of()
    rooms = [within() for _ in range(4)]
    y, h, dres, dx = (v for _, v in rooms)
    R.rms_norm_dropout(x, res, p, rng, w, out=y, residual_out=h)
    keep = ref.kept(rows, hidden, p, SEED, OFFSET)
    want = ref.forward_h(x, res, keep, p).to(DEV)
    fine = torch.arange(rows, device=DEV) != 4
    assert torch.equal(h, want)
    assert_within(y[fine], *ref.norm(want[fine], w, 1e-6, 0.0), "y")

    h[4] = src[1][3]   # the gradient's rows are finite, but one of dy, which is left out of dw's
    dy[4] = float("nan")
    _, _, dw = R.rms_norm_dropout_backward(dy, h, p, rng, w, dh, dresidual=dres, dx=dx)
    keep = keep.to(DEV)
    want = ref.backward(dy[fine], h[fine], w, dh[fine], keep[fine], p, 1e-6, 0.0)
    assert_within(dres[fine], want[0], want[1], "dresidual")
    assert_within(dx[fine], want[2], want[3], "dx")
    assert bool(dw.isnan().all())
    dy[4] = 0.0
    only, dw = R.rms_norm_backward(dy, h, w)
    want = ref.backward(dy, h, w, None, None, 0.0, 1e-6, 0.0)
    assert_within(only, want[0], want[1], "dx alone")
    assert_within(dw, want[4], want[5], "dw")
    for room, _ in rooms:
        assert bool((room[rows * hidden:] == 7.5).all())
    # from a place off the boundary, element by element
    off = torch.empty(rows * hidden + 1, dtype=t, device=DEV)[1:].view(rows, hidden)
    y2, h2 = R.rms_norm_dropout(off.copy_(x), res, p, rng, w)
    same = R.rms_norm_dropout(x, res, p, rng, w)[1]
    assert torch.equal(h2[fine], same[fine])
    assert_within(y2[fine], *ref.norm(h2[fine], w, 1e-6, 0.0), "y, element by element")
    off.copy_(dy)
    two, dw2 = R.rms_norm_backward(off, h, w)
    assert_within(two, want[0], want[1], "dx alone, element by element")
    assert_within(dw2, want[4], want[5], "dw, element by element")
