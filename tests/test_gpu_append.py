"""The append of keys and values to a paged cache, with the head norm and the
rotation on the way, against the formulas in 64 bits (GB300 only).

Tolerances: values as in rope_ref.py; an E4M3 code stands for a value within
half a step (2^-4 relative, 2^-10 absolute below the smallest normal) of the
exact quotient, saturated at 448; values that are only stored are exact."""
import pytest
import torch

import rope_ref as ref
from test_gpu_rope import DEV, T, freqs, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R
    from row_reduction_norm_gb300 import _native as N


def make(dtype, cache, lens, news, pad, q, k, d, page, heads_first, seed, spare=3):
    """A batch, its pages in random order, and caches filled with noise."""
    g = gen(seed)
    need = [-(-(a + b) // page) for a, b in zip(lens, news)]
    pages = sum(need) + spare
    order = torch.randperm(pages, device=DEV, generator=g).int()
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m].cpu()
        at += m
    total = sum(news)
    qkv = normal(g, total + pad, (q + 2 * k) * d, dtype=T[dtype])
    cu = torch.tensor([0] + torch.tensor(news).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    caches = []
    for _ in range(2):
        shape = (pages, k, page, d) if heads_first else (pages, page, k, d)
        if cache == "e4m3":
            c = torch.randint(0, 255, shape, device=DEV, generator=g, dtype=torch.uint8)
            c = torch.where((c & 127) == 127, c - 1, c).view(torch.float8_e4m3fn)
        else:
            c = normal(g, *shape, dtype=T[dtype])
        caches.append(c.permute(0, 2, 1, 3) if heads_first else c)
    return g, qkv, caches, table.to(DEV), cu, torch.tensor(lens, dtype=torch.int32, device=DEV), total


def slots(lens, news, table, page):
    at = torch.cat([torch.arange(a, a + b) for a, b in zip(lens, news)])
    t = table.cpu().long()
    pages = torch.cat([t[i][torch.arange(a, a + b) // page] for i, (a, b) in enumerate(zip(lens, news))])
    return at.to(DEV), pages.to(DEV), (at % page).to(DEV)


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def check_cache(cache, before, pages, rows, want, bound, scale, what):
    if cache.dtype == torch.float8_e4m3fn:
        w = (want / scale).clamp(-448.0, 448.0)
        bound = bound / scale + torch.maximum(w.abs() * 2.0 ** -4, torch.full_like(w, 2.0 ** -10))
        want = w
    got = cache.float()[pages, rows]
    ref.assert_within(got, want, bound, what)
    a, b = bits(cache).clone(), bits(before).clone()
    a[pages, rows] = 0
    b[pages, rows] = 0
    assert torch.equal(a, b), f"{what}: a row outside the batch was written"


CASES = [
    # lens, news, pad, q, k, d, rot, page, heads_first
    ([0], [1], 0, 4, 1, 128, 128, 16, False),
    ([5, 0, 31, 16, 0], [1, 1, 1, 1, 1], 0, 8, 2, 128, 128, 16, False),
    ([0, 7, 0, 100, 3], [33, 0, 1, 64, 5], 4, 5, 3, 64, 64, 16, True),
    ([3, 0], [20, 0], 1, 3, 1, 96, 48, 7, False),
    ([0, 0, 0], [0, 0, 9], 2, 0, 2, 80, 20, 1, True),
    ([11] * 40, [3] * 40, 0, 2, 2, 72, 72, 5, False),
    ([2, 1], [130, 77], 9, 7, 1, 48, 14, 64, False),
    ([1000], [257], 0, 4, 4, 256, 64, 128, True),
]


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(dtype, cache, interleaved, case):
    lens, news, pad, q, k, d, rot, page, heads_first = CASES[case]
    norm = case % 3 != 2
    g, qkv, (kc, vc), table, cu, cl, n = make(dtype, cache, lens, news, pad, q, k, d, page, heads_first, case)
    qw = normal(g, d, dtype=T[dtype], std=0.2, mean=1.0) if norm else None
    kw = normal(g, d, dtype=T[dtype], std=0.2, mean=1.0) if norm else None
    ks, vs = (0.05, 0.03) if cache == "e4m3" else (1.0, 1.0)
    f = freqs(rot)
    k0, v0, x0 = kc.clone(), vc.clone(), qkv.clone()
    q_out = torch.full((n + pad, q * d), -7.0, dtype=T[dtype], device=DEV) if q else None
    dropped = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, q_w=qw, k_w=kw, norm=norm, interleaved=interleaved,
                       k_scale=ks, v_scale=vs, q_out=q_out, dropped=dropped)
    assert got is q_out and int(dropped) == 0 and torch.equal(qkv, x0)
    assert torch.equal(cl, torch.tensor(lens, dtype=torch.int32, device=DEV))
    at, pages, rows = slots(lens, news, table, page)
    theta = ref.phases(at[None], f, (rot // 2,))
    y, bound = ref.forward(qkv[:n], q, k, d, theta, rot, interleaved, qw, kw, 1e-6, 0.0, norm)
    if q:
        ref.assert_within(q_out[:n], y[:, :q].reshape(n, -1), bound[:, :q].reshape(n, -1), "q_out")
        assert bool((q_out[n:] == -7.0).all())
    check_cache(kc, k0, pages, rows, y[:, q:], bound[:, q:], ks, "keys")
    v = qkv[:n].view(n, q + 2 * k, d)[:, q + k:]
    if cache != "e4m3":
        assert torch.equal(vc[pages, rows], v), "values are stored as they are"
    check_cache(vc, v0, pages, rows, v.double(), torch.zeros_like(v, dtype=torch.float64) + 4e-7 * v.double().abs(), vs,
                "values")


def test_given_positions_with_axes_and_in_place_queries():
    lens, news, q, k, d, page, sections = [4, 0, 9], [5, 8, 1], 4, 2, 64, 16, (8, 12, 12)
    g, qkv, (kc, vc), table, cu, cl, n = make("bf16", "bf16", lens, news, 0, q, k, d, page, False, 1)
    pos = torch.randint(0, 300, (3, n), device=DEV, generator=g).int()
    f = freqs(64)
    keep = qkv.clone()
    y, bound = ref.forward(qkv, q, k, d, ref.phases(pos, f, sections), 64, False, None, None, 1e-6, 0.0, True)
    k0 = kc.clone()
    R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, positions=pos, sections=sections, q_out=qkv)
    ref.assert_within(qkv[:, :q * d], y[:, :q].reshape(n, -1), bound[:, :q].reshape(n, -1), "queries in place")
    assert torch.equal(qkv[:, q * d:], keep[:, q * d:])
    _, pages, rows = slots(lens, news, table, page)
    check_cache(kc, k0, pages, rows, y[:, q:], bound[:, q:], 1.0, "keys")


def test_append_agrees_with_the_rotary_call():
    """Queries and keys have the bits that qk_norm_rope gives them."""
    lens, news, q, k, d, page = [40, 3], [17, 30], 8, 2, 128, 16
    g, qkv, (kc, vc), table, cu, cl, n = make("bf16", "bf16", lens, news, 0, q, k, d, page, False, 2)
    qw, kw = normal(g, d, dtype=torch.bfloat16), normal(g, d, dtype=torch.bfloat16)
    f = freqs(128)
    at, pages, rows = slots(lens, news, table, page)
    y = R.qk_norm_rope(qkv, q, k, d, at, f, q_w=qw, k_w=kw)
    q_out = R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, q_w=qw, k_w=kw)
    assert torch.equal(q_out, y[:, :q * d])
    assert torch.equal(kc[pages, rows].reshape(n, -1), y[:, q * d:])


def test_missing_pages_are_skipped_and_counted():
    """Absent pages, page numbers outside the cache, rows past the page table
    and a negative length: nothing is written for them, the queries are."""
    lens, news, q, k, d, page = [0, 14, 5, 2, 0], [20, 4, 3, 2, 1], 4, 2, 64, 16
    g, qkv, (kc, vc), table, cu, cl, n = make("bf16", "bf16", lens, news, 0, q, k, d, page, False, 3)
    full_at, pages, rows = slots(lens, news, table, page)
    f = freqs(64)
    table[0, 1] = -1                  # tokens 16 .. 19 of sequence 0
    table[1, 0] = kc.shape[0]         # rows 14 and 15 of sequence 1: one past the last page
    table[2, 0] = 2 ** 31 - 1         # all three of sequence 2
    cl[3] = table.shape[1] * page     # both of sequence 3: past its page table
    cl[4] = -5                        # a negative row
    ok = torch.ones(n, dtype=torch.bool, device=DEV)
    ok[16:20] = False
    ok[20:22] = False
    ok[24:30] = False
    k0, v0 = kc.clone(), vc.clone()
    dropped = torch.full((1,), 5, dtype=torch.int32, device=DEV)
    q_out = R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, dropped=dropped)
    torch.cuda.synchronize()
    assert int(dropped) == 5 + int((~ok).sum())
    at = full_at.clone()
    at[27:29] = int(cl[3]) + torch.arange(2, device=DEV)
    at[29] = -5
    y, bound = ref.forward(qkv, q, k, d, ref.phases(at[None], f, (32,)), 64, False, None, None, 1e-6, 0.0, True)
    ref.assert_within(q_out, y[:, :q].reshape(n, -1), bound[:, :q].reshape(n, -1), "queries")
    check_cache(kc, k0, pages[ok], rows[ok], y[ok][:, q:], bound[ok][:, q:], 1.0, "keys")
    v = qkv.view(n, q + 2 * k, d)[ok][:, q + k:].double()
    check_cache(vc, v0, pages[ok], rows[ok], v, v * 0, 1.0, "values")


def test_special_values_in_an_8bit_cache():
    d = 64
    g, qkv, (kc, vc), table, cu, cl, n = make("f32", "e4m3", [0], [4], 0, 1, 1, d, 16, False, 4)
    x = qkv.view(4, 3, d)
    x[:, 2] = 0.0
    x[0, 2, :6] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e9, 2.0 ** -9, 2.0 ** -11], device=DEV)
    R.qkv_append(qkv, kc, vc, table, cu, cl, 1, 1, d, freqs(d), norm=False)
    _, pages, rows = slots([0], [4], table, 16)
    got = vc.float()[pages, rows][0, 0, :6]
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and got[3] == 448
    assert got[4] == 2.0 ** -9 and got[5] == 0


def test_offsets_past_32_bits():
    """A cache of 2^31 + elements: the last pages are reached."""
    k, d, page = 1, 128, 64
    pages = (2 ** 31) // (page * d) + 5
    kc = torch.zeros(pages, page, k, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    g = gen(8)
    qkv = normal(g, 3, 4 * d, dtype=torch.bfloat16)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    cl = torch.tensor([62], dtype=torch.int32, device=DEV)
    R.qkv_append(qkv, kc, vc, table, cu, cl, 2, k, d, freqs(d), norm=False)
    v = qkv.view(3, 4, d)[:, 3]
    assert torch.equal(vc[pages - 1, 62:, 0], v[:2]) and torch.equal(vc[pages - 2, 0, 0], v[2])
    assert int((vc != 0).any(-1).sum()) == 3 and int((kc != 0).any(-1).sum()) == 3


def test_captured_step_with_padding():
    """A captured step of 8 slots replayed with fewer tokens and other lengths."""
    q, k, d, page, slots_n = 8, 2, 128, 16, 8
    g, qkv, (kc, vc), table, cu, cl, n = make("bf16", "bf16", [30] * slots_n, [1] * slots_n, 0, q, k, d, page, False, 5)
    f = freqs(d)
    q_out = torch.zeros(n, q * d, dtype=torch.bfloat16, device=DEV)
    R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, q_out=q_out)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, q_out=q_out)
    lens, news = [3, 0, 17, 31, 8, 0, 0, 0], [1, 2, 0, 1, 1, 0, 0, 0]
    cl.copy_(torch.tensor(lens))
    cu.copy_(torch.tensor([0] + torch.tensor(news).cumsum(0).tolist()))
    qkv.copy_(normal(g, *qkv.shape, dtype=qkv.dtype))
    q_out.fill_(-7.0)
    k0 = kc.clone()
    gr.replay()
    torch.cuda.synchronize()
    n = sum(news)
    at, pages, rows = slots(lens, news, table, page)
    y, bound = ref.forward(qkv[:n], q, k, d, ref.phases(at[None], f, (64,)), 128, False, None, None, 1e-6, 0.0, True)
    ref.assert_within(q_out[:n], y[:, :q].reshape(n, -1), bound[:, :q].reshape(n, -1), "queries")
    assert bool((q_out[n:] == -7.0).all())
    check_cache(kc, k0, pages, rows, y[:, q:], bound[:, q:], 1.0, "keys")


def test_python_refusals():
    lens, news, q, k, d = [0], [2], 2, 1, 64
    g, qkv, (kc, vc), table, cu, cl, n = make("bf16", "bf16", lens, news, 0, q, k, d, 16, False, 6)
    f = freqs(d)
    ok = dict(k_cache=kc, v_cache=vc, page_table=table, cu_tokens=cu, cache_lens=cl)
    for bad in (dict(k_cache=kc[..., :32]), dict(v_cache=vc[:1]), dict(k_cache=kc.float(), v_cache=vc.float()),
                dict(page_table=table.long()), dict(page_table=table[0]), dict(cu_tokens=cu[:1]),
                dict(cu_tokens=cu.long()), dict(cache_lens=cl.cpu()), dict(k_cache=kc.cpu(), v_cache=vc.cpu())):
        with pytest.raises((ValueError, TypeError, N.RmsNormError)):
            a = {**ok, **bad}
            R.qkv_append(qkv, a["k_cache"], a["v_cache"], a["page_table"], a["cu_tokens"], a["cache_lens"], q, k, d, f)
    with pytest.raises((ValueError, N.RmsNormError)):
        R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, sections=(16, 16))
    with pytest.raises(ValueError):
        R.qkv_append(qkv, kc, vc, table, cu, cl, q, k, d, f, q_out=torch.empty(1, q * d, device=DEV, dtype=qkv.dtype))
