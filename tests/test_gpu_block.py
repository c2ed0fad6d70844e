"""The operators in a row, as a transformer block uses them (GB300 only): a
training step's attention half with its gradients, and a served batch that
fills and reads a paged cache, against the whole formula in 64 bits.

Tolerance, of the norm of a result: every operator and product here is off by
at most 64 u or K u (K = 256 terms, u = 2^-24) of the sizes of its terms, at
most 1.6e-5; ten of them in a row, each able to raise what came before by the
ratio of the terms' sizes to their sum (under 2 in norm for these random
inputs): 2 x 10 x 1.6e-5 = 3.2e-4."""
import pytest
import torch

import drop_ref
import rope_ref
from test_gpu_rope import DEV, freqs, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R

TOL = 3.2e-4
HIDDEN, Q, K, D = 256, 4, 2, 64


def near(got, want, what):
    off = float((got.double() - want).norm() / want.norm())
    assert off <= TOL, f"{what}: {off:.3g} of its norm off"


def attention(q, k, v):
    """Causal attention of one sequence, [tokens, heads, D] each, shared key heads."""
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
    n, m = s.shape[-2:]
    i = torch.arange(n, device=q.device)[:, None] + (m - n)
    s = s.masked_fill(torch.arange(m, device=q.device)[None] > i, float("-inf"))
    return torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v).flatten(1)


def test_training_step_with_its_gradients():
    n, p, eps = 50, 0.1, 1e-6
    g = gen(17)
    f32 = torch.float32
    x, res = normal(g, n, HIDDEN, dtype=f32), normal(g, n, HIDDEN, dtype=f32)
    w, qw, kw = (normal(g, m, dtype=f32, std=0.1, mean=1.0) for m in (HIDDEN, D, D))
    wide = (Q + 2 * K) * D
    w_in = normal(g, HIDDEN, wide, dtype=f32, std=HIDDEN ** -0.5)
    w_out = normal(g, Q * D, HIDDEN, dtype=f32, std=(Q * D) ** -0.5)
    to, th = normal(g, n, HIDDEN, dtype=f32), normal(g, n, HIDDEN, dtype=f32)   # gradients of the two results
    rng = torch.tensor([99, 7], device=DEV)
    f, pos = freqs(D), torch.arange(n, device=DEV)

    # the framework's calls, products and attention by torch
    y, h = R.rms_norm_dropout(x, res, p, rng, w=w, eps=eps)
    qkv = y @ w_in
    qk = R.qk_norm_rope(qkv, Q, K, D, pos, f, q_w=qw, k_w=kw, eps=eps)
    leaves = [t.detach().clone().requires_grad_() for t in (qk, qkv[:, (Q + K) * D:])]
    heads = leaves[0].view(n, Q + K, D)
    o = attention(heads[:, :Q], heads[:, Q:], leaves[1].view(n, K, D))
    out = o.detach() @ w_out
    dqk, dv = torch.autograd.grad(o, leaves, to @ w_out.t())
    dqkv = torch.empty_like(qkv)
    dqkv[:, (Q + K) * D:] = dv
    _, dqw, dkw = R.qk_norm_rope_backward(dqk, qkv, Q, K, D, pos, f, q_w=qw, k_w=kw, eps=eps, out=dqkv)
    dres, dx, dw = R.rms_norm_dropout_backward(dqkv @ w_in.t(), h, p, rng, w=w, dresidual_out=th, eps=eps)
    got = {"x": dx, "residual": dres, "w": dw, "q_w": dqw, "k_w": dkw, "w_in": y.t() @ dqkv, "w_out": o.detach().t() @ to}

    # the same in 64 bits
    keep = drop_ref.kept(n, HIDDEN, p, 99, 7).to(DEV)
    v = {k: t.double().requires_grad_() for k, t in
         {"x": x, "residual": res, "w": w, "q_w": qw, "k_w": kw, "w_in": w_in, "w_out": w_out}.items()}
    h64 = v["residual"] + torch.where(keep, v["x"] * (65536 / (65536 - drop_ref.threshold(p))), torch.zeros_like(v["x"]))
    y64 = h64 / torch.sqrt((h64 * h64).mean(-1, keepdim=True) + eps) * v["w"]
    packed = (y64 @ v["w_in"]).view(n, Q + 2 * K, D)
    normed = torch.cat((rope_ref.head_norm(packed[:, :Q], v["q_w"], 0.0, eps, True),
                        rope_ref.head_norm(packed[:, Q:Q + K], v["k_w"], 0.0, eps, True)), 1)
    theta = rope_ref.phases(pos[None], f, (D // 2,))
    c, s = torch.cos(theta)[:, None], torch.sin(theta)[:, None]
    a, b = normed[..., :D // 2], normed[..., D // 2:]
    turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    o64 = attention(turned[:, :Q], turned[:, Q:], packed[:, Q + K:])
    out64 = o64 @ v["w_out"]
    near(h, h64.detach(), "residual_out")
    near(out, out64.detach(), "output")
    grads = torch.autograd.grad((out64 * to.double()).sum() + (h64 * th.double()).sum(), list(v.values()))
    for (name, _), want in zip(v.items(), grads):
        near(got[name], want, f"gradient of {name}")


def test_served_batch_fills_and_reads_a_paged_cache():
    """Three prompts of different lengths, then four steps of one token each,
    with padding rows throughout; each attention reads its pages."""
    page, prompts, steps, eps = 16, [21, 1, 40], 4, 1e-6
    g = gen(23)
    f32 = torch.float32
    w, qw, kw = (normal(g, m, dtype=f32, std=0.1, mean=1.0) for m in (HIDDEN, D, D))
    w_in = normal(g, HIDDEN, (Q + 2 * K) * D, dtype=f32, std=HIDDEN ** -0.5)
    f = freqs(D)
    need = [-(-(p + steps) // page) for p in prompts]
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).int()
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    table = table.to(DEV)
    kc, vc = (torch.zeros(sum(need), page, K, D, device=DEV) for _ in range(2))
    hidden = [normal(g, p + steps, HIDDEN, dtype=f32) for p in prompts]   # every token's input, known beforehand

    # what each token's attention gives, in 64 bits over the whole sequence
    want = []
    for i, xs in enumerate(hidden):
        n = len(xs)
        z = xs.double()
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * w.double()
        packed = (z @ w_in.double()).view(n, Q + 2 * K, D)
        theta = rope_ref.phases(torch.arange(n, device=DEV)[None], f, (D // 2,))
        turned, _ = rope_ref.rotate(
            torch.cat((rope_ref.head_norm(packed[:, :Q], qw.double(), 0.0, eps, True),
                       rope_ref.head_norm(packed[:, Q:Q + K], kw.double(), 0.0, eps, True)), 1), theta, D, D, False)
        want.append(attention(turned[:, :Q], turned[:, Q:], packed[:, Q + K:]))

    lens = [0, 0, 0]
    dropped = torch.zeros(1, dtype=torch.int32, device=DEV)
    for step in range(1 + steps):
        news = prompts if step == 0 else [1, 1, 1]
        total, pad = sum(news), 5
        rows = torch.zeros(total + pad, HIDDEN, device=DEV)
        rows[:total] = torch.cat([hidden[i][lens[i]:lens[i] + news[i]] for i in range(3)])
        qkv = R.rms_norm(rows, w=w, eps=eps) @ w_in
        cu = torch.tensor([0, news[0], news[0] + news[1], total], dtype=torch.int32, device=DEV)
        q_out = R.qkv_append(qkv, kc, vc, table, cu, torch.tensor(lens, dtype=torch.int32, device=DEV), Q, K, D, f,
                             q_w=qw, k_w=kw, eps=eps, dropped=dropped)
        first = 0
        for i in range(3):
            n = lens[i] + news[i]
            pages = table[i, :need[i]].long()
            k, v = (c[pages].reshape(-1, K, D)[:n] for c in (kc, vc))
            o = attention(q_out[first:first + news[i]].view(-1, Q, D), k, v)
            near(o, want[i][lens[i]:n], f"step {step}, sequence {i}")
            first += news[i]
            lens[i] = n
    assert int(dropped) == 0
