"""The rotary, append and dropout operators at the ends of what they take
(GB300 only): token rows far apart, tensors past 32-bit offsets, batches that
give a block more tokens than it looks up at once, several threads, weights
off every boundary, and the two ways a Python call is made.

What is compared bit for bit is the same arithmetic on the same values; other
tolerances are those of rope_ref.py and drop_ref.py."""
import threading

import numpy as np
import pytest
import torch

import drop_ref
import rope_ref as ref
from test_gpu_rope import DEV, T, freqs, gen, inputs, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R

SEED, OFFSET = 0x123456789ABCDEF, 77


def spread(t, stride):
    """The rows of t, `stride` elements apart."""
    rows, width = t.shape
    out = torch.empty((rows - 1) * stride + width, dtype=t.dtype, device=DEV).as_strided((rows, width), (stride, 1))
    out.copy_(t)
    return out


# whole heads, heads through shared memory, heads in narrow pieces
@pytest.mark.parametrize("d,rot", [(128, 128), (80, 20), (34, 34)])
def test_token_rows_far_apart(d, rot):
    """Rows more than 2^28 bytes apart, 5 GB in all."""
    tokens, q, k, far = 20, 3, 2, 2 ** 27 + 64
    g, qkv, pos, f, qw, kw = inputs("bf16", tokens, q, k, d, rot, (rot // 2,), 5, extra=0)
    x = spread(qkv, far)
    out = spread(torch.zeros_like(qkv), far)
    want = R.qk_norm_rope(qkv, q, k, d, pos, f, qw, kw)
    assert torch.equal(R.qk_norm_rope(x, q, k, d, pos, f, qw, kw, out=out), want)
    dy = normal(g, tokens, (q + k) * d, dtype=torch.bfloat16)
    dx, dq, dk = R.qk_norm_rope_backward(spread(dy, far), x, q, k, d, pos, f, qw, kw, out=out)
    near = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, qw, kw)
    assert torch.equal(dx, near[0])
    theta = ref.phases(pos, f, (rot // 2,))
    want = ref.backward(dy, qkv, q, k, d, theta, rot, False, qw, kw, 1e-6, 0.0, True)
    ref.assert_within(dq, want[2], want[3], "dq_w")
    ref.assert_within(dk, want[4], want[5], "dk_w")


def test_append_of_rows_far_apart():
    tokens, q, k, d, far = 20, 2, 1, 128, 2 ** 27 + 64
    g, qkv, pos, f, qw, kw = inputs("bf16", tokens, q, k, d, d, (d // 2,), 6, extra=1)
    caches = [torch.zeros(2, 2, 16, k, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = [R.qkv_append(x, c[0], c[1], table, cu, lens, q, k, d, f, q_w=qw, k_w=kw)
           for x, c in zip((qkv, spread(qkv, far)), caches)]
    assert torch.equal(*got) and torch.equal(*caches) and int((caches[0] != 0).any(-1).sum()) == 2 * tokens


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("d,rot", [(64, 64), (80, 20)])
def test_append_of_many_tokens(d, rot, cache):
    """More tokens than the blocks look up at once, in sequences of 0 to some thousands."""
    tokens, q, k, page, seqs = 60000, 1, 1, 16, 37
    g, qkv, _, f, qw, kw = inputs("bf16", tokens, q, k, d, rot, (rot // 2,), 7, extra=1)
    cuts = torch.sort(torch.randint(0, tokens, (seqs - 1,), device=DEV, generator=g)).values
    cuts[5] = cuts[6] = cuts[4]
    cu = torch.cat((torch.zeros_like(cuts[:1]), torch.sort(cuts).values, torch.full_like(cuts[:1], tokens)))
    news = cu.diff()
    lens = torch.randint(0, 40, (seqs,), device=DEV, generator=g)
    need = -(-(lens + news) // page)
    first = torch.cat((torch.zeros_like(need[:1]), need.cumsum(0)))
    total = int(first[-1])
    order = torch.randperm(total, device=DEV, generator=g).int()
    most = int(need.max())
    at = torch.arange(most, device=DEV)[None] + first[:-1, None]
    table = torch.where(at < first[1:, None], order[at.clamp(max=total - 1)], torch.full_like(at, -1).int())
    kind = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    kc, vc = (torch.zeros(total, page, k, d, device=DEV).to(kind) for _ in range(2))
    got = R.qkv_append(qkv, kc, vc, table.int(), cu.int(), lens.int(), q, k, d, f, q_w=qw, k_w=kw)

    seq = torch.repeat_interleave(torch.arange(seqs, device=DEV), news)
    index = torch.arange(tokens, device=DEV) - cu[seq] + lens[seq]
    both = R.qk_norm_rope(qkv, q, k, d, index, f, qw, kw)
    assert torch.equal(got, both[:, :q * d])
    pages = table[seq, index // page].long()
    key, value = kc[pages, index % page, 0], vc[pages, index % page, 0]
    if cache == "same":
        assert torch.equal(key, both[:, q * d:]) and torch.equal(value, qkv[:, 2 * d:])
    else:
        # a value that is only stored has one rounding, the codes' own
        assert torch.equal(value.view(torch.uint8), qkv[:, 2 * d:].to(kind).view(torch.uint8))
        theta = ref.phases(index[None], f, (rot // 2,))
        want, bound = ref.forward(qkv, q, k, d, theta, rot, False, qw, kw, 1e-6, 0.0, True)
        step = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10))
        ref.assert_within(key.float()[:, None], want[:, q:], (bound + step)[:, q:], "keys")


@pytest.mark.parametrize("hidden,rows", [(8192, 262144 + 9), (2047, 1049088 + 9), (65536, 32768 + 9)])
def test_dropout_past_32_bit_offsets(hidden, rows):
    """2^31 elements and some rows more, the last rows looked at; in place."""
    last, p, t = 9, 0.25, torch.bfloat16
    g = gen(hidden)
    x, res = (torch.zeros(rows, hidden, dtype=t, device=DEV) for _ in range(2))
    w = normal(g, hidden, dtype=t, std=0.2, mean=1.0)
    for v in (x, res):
        v[-last:] = normal(g, last, hidden, dtype=t)
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device=DEV)
    keep = drop_ref.kept(last, hidden, p, SEED, OFFSET, first=rows - last)
    h = drop_ref.forward_h(x[-last:], res[-last:], keep, p)
    R.rms_norm_dropout(x, res, p, rng, w, out=x, residual_out=res)
    assert torch.equal(res[-last:].cpu(), h)
    ref.assert_within(x[-last:].cpu(), *drop_ref.norm(h, w.cpu(), 1e-6, 0.0), "y")
    assert not bool(x[-last - 1].any())

    dy = x
    want = drop_ref.backward(dy[-last:].cpu(), h, w.cpu(), None, keep, p, 1e-6, 0.0)
    _, _, dw = R.rms_norm_dropout_backward(dy, res, p, rng, w, dresidual=x, dx=res)
    ref.assert_within(x[-last:].cpu(), want[0], want[1], "dresidual")
    ref.assert_within(res[-last:].cpu(), want[2], want[3], "dx")
    ref.assert_within(dw.cpu(), want[4], want[5], "dw")


def test_weights_off_every_boundary():
    """Where the head weights start has no part in the result."""
    tokens, q, k, d = 50, 4, 2, 128
    g, qkv, pos, f, qw, kw = inputs("bf16", tokens, q, k, d, d, (d // 2,), 9)
    flat = torch.zeros(4 * d, dtype=torch.bfloat16, device=DEV)
    q2, k2 = flat[1:1 + d], flat[2 * d + 3:3 * d + 3]
    q2.copy_(qw), k2.copy_(kw)
    dy = normal(g, tokens, (q + k) * d, dtype=torch.bfloat16)
    assert torch.equal(R.qk_norm_rope(qkv, q, k, d, pos, f, q2, k2), R.qk_norm_rope(qkv, q, k, d, pos, f, qw, kw))
    for a, b in zip(R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, q2, k2),
                    R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, qw, kw)):
        assert torch.equal(a, b)


def calls(seed, stream=None, kind=int):
    """Every operator once, on inputs that follow from the seed."""
    tokens, q, k, d, rows, hidden = 40, kind(4), kind(2), kind(64), 50, 1024
    g, qkv, pos, f, qw, kw = inputs("bf16", tokens, 4, 2, 64, 64, (32,), seed, extra=2)
    dy = normal(g, tokens, 6 * 64, dtype=torch.bfloat16)
    x, res, dn, dh = (normal(g, rows, hidden, dtype=torch.bfloat16) for _ in range(4))
    w = normal(g, hidden, dtype=torch.bfloat16, mean=1.0)
    rng = torch.tensor([seed, 3], dtype=torch.int64, device=DEV)
    kc, vc = (torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    on = {} if stream is None else {"stream": stream}
    y, h = R.rms_norm_dropout(x, res, 0.1, rng, w, **on)
    out = [R.qk_norm_rope(qkv, q, k, d, pos, f, qw, kw, **on),
           *R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, qw, kw, **on),
           R.qkv_append(qkv, kc, vc, ints(2, 0, 1, 3).view(2, 2), ints(0, 21, 40), ints(5, 0), q, k, d, f, q_w=qw,
                        k_w=kw, **on), kc, vc, y, h,
           *R.rms_norm_dropout_backward(dn, h, 0.1, rng, w, dh, **on), *R.rms_norm_backward(dn, h, w, dh, **on)]
    return out


def test_both_ways_of_a_call_agree():
    """Natively and through the Python bodies (a stream given, counts of another integer type)."""
    plain = calls(11)
    for other in (calls(11, torch.cuda.current_stream()), calls(11, kind=np.int64)):
        assert len(other) == len(plain)
        for a, b in zip(plain, other):
            assert torch.equal(a, b)


def test_threads_on_their_own_streams():
    want = [calls(s) for s in range(4)]
    torch.cuda.synchronize()
    errors = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    for a, b in zip(calls(s), want[s]):
                        if not torch.equal(a, b):
                            errors.append(s)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


# a token's heads in slices over the blocks: whole pieces, narrow ones, heads through shared memory
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,q,k", [(1, 48, 12), (2, 5, 64), (7, 64, 0), (29, 33, 31), (151, 40, 9)])
@pytest.mark.parametrize("d,rot", [(128, 128), (72, 48), (80, 20), (34, 34)])
def test_few_tokens_of_many_heads(dtype, tokens, q, k, d, rot):
    g, qkv, pos, f, qw, kw = inputs(dtype, tokens, q, k, d, rot, (rot // 2,), tokens + d)
    dy = normal(g, tokens, (q + k) * d, dtype=T[dtype])
    theta = ref.phases(pos, f, (rot // 2,))
    y = R.qk_norm_rope(qkv, q, k, d, pos, f, qw, kw)
    ref.assert_within(y, *ref.forward(qkv, q, k, d, theta, rot, False, qw, kw, 1e-6, 0.0, True), "y")
    got = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, qw, kw)
    want = ref.backward(dy, qkv, q, k, d, theta, rot, False, qw, kw, 1e-6, 0.0, True)
    for i, name in enumerate(("dx", "dq_w", "dk_w")):
        ref.assert_within(got[i], want[2 * i], want[2 * i + 1], name)
    dx = R.qk_norm_rope_backward(dy, None, q, k, d, pos, f, norm=False, out=dy)[0]   # in place
    assert dx is dy
    back = ref.rotate(want[0].new_tensor(0.0) + y.double().reshape(tokens, q + k, d), theta, d, rot, False, back=True)
    again = R.qk_norm_rope_backward(y, None, q, k, d, pos, f, norm=False)[0]
    ref.assert_within(again, back[0], 32 * ref.U * back[1] + ref.half_step(T[dtype]) * (1 + 32 * ref.U) * back[0].abs(),
                      "turned back")


# around the row and token counts from which a weight's gradient takes a second launch
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hidden", [40, 192, 832, 2048, 8192, 201, 2051, 20480])
def test_weight_gradients_of_few_rows(dtype, hidden):
    t, g, p = T[dtype], gen(hidden), 0.25
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device=DEV)
    w = normal(g, hidden, dtype=t, std=0.2, mean=1.0)
    ws = torch.full((R.rmsnorm_bwd_workspace_bytes(600, hidden, {"f32": 0, "bf16": 1}[dtype]),), 255, dtype=torch.uint8,
                    device=DEV)   # NaN where nothing is written
    for rows in (1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 256, 257):
        dy, h, dh = (normal(g, rows, hidden, dtype=t) for _ in range(3))
        keep = drop_ref.kept(rows, hidden, p, SEED, OFFSET).to(DEV)
        want = drop_ref.backward(dy, h, w, dh, keep, p, 1e-6, 0.0)
        got = R.rms_norm_dropout_backward(dy, h, p, rng, w, dh, workspace=ws)
        for i, name in enumerate(("dresidual", "dx", "dw")):
            ref.assert_within(got[i], want[2 * i], want[2 * i + 1], f"{name}, {rows} rows")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q,k,d,rot", [(4, 2, 64, 64), (24, 8, 96, 96), (0, 3, 80, 20), (5, 0, 34, 34)])
def test_weight_gradients_of_few_tokens(dtype, q, k, d, rot):
    for tokens in (1, 2, 7, 8, 9, 16, 40, 64, 65, 129, 304):
        g, qkv, pos, f, qw, kw = inputs(dtype, tokens, q, k, d, rot, (rot // 2,), tokens)
        dy = normal(g, tokens, (q + k) * d, dtype=T[dtype])
        theta = ref.phases(pos, f, (rot // 2,))
        want = ref.backward(dy, qkv, q, k, d, theta, rot, False, qw, kw, 1e-6, 0.0, True)
        ws = torch.full((R.rmsnorm_qk_rope_bwd_workspace_bytes(d),), 255, dtype=torch.uint8, device=DEV)
        got = R.qk_norm_rope_backward(dy, qkv, q, k, d, pos, f, qw, kw, workspace=ws)
        for i, name in enumerate(("dx", "dq_w", "dk_w")):
            ref.assert_within(got[i], want[2 * i], want[2 * i + 1], f"{name}, {tokens} tokens")


def test_small_gradients_in_a_graph():
    """Calls of one cluster and of two launches, one after another on one
    workspace, replayed on new inputs; two graphs on two streams."""
    g = gen(12)
    q, k, d = 4, 2, 64
    f, qw, kw = freqs(d), normal(g, d, dtype=torch.bfloat16, mean=1.0), normal(g, d, dtype=torch.bfloat16, mean=1.0)
    sizes = [(3, 9), (200, 700), (1, 30), (64, 2)]
    sets = []
    for _ in range(2):
        ws = torch.empty(8 << 20, dtype=torch.uint8, device=DEV)
        one = [dict(x=normal(g, a, (q + k) * d, dtype=torch.bfloat16), dy=normal(g, a, (q + k) * d, dtype=torch.bfloat16),
                    pos=torch.arange(a, device=DEV), h=normal(g, b, 832, dtype=torch.bfloat16),
                    dh=normal(g, b, 832, dtype=torch.bfloat16)) for a, b in sizes]
        sets.append((ws, one))
    w = normal(g, 832, dtype=torch.bfloat16, mean=1.0)

    def run(ws, one):
        out = []
        for s in one:
            out += R.qk_norm_rope_backward(s["dy"], s["x"], q, k, d, s["pos"], f, qw, kw, workspace=ws)
            out += R.rms_norm_backward(s["dh"], s["h"], w, workspace=ws)
        return out

    for s in sets:
        run(*s)
    graphs = []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, run(*s)))
    streams = [torch.cuda.Stream() for _ in sets]
    for turn in range(3):
        for _, one in sets:
            for s in one:
                for name in ("x", "dy", "h", "dh"):
                    s[name].copy_(normal(g, *s[name].shape, dtype=torch.bfloat16))
        torch.cuda.synchronize()
        for s, (gr, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for s, (_, got) in zip(sets, graphs):
            for a, b in zip(run(*s), got):
                assert torch.equal(a, b)
