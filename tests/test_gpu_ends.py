"""The operators at the two ends of a model as they are used (GB300 only): a
training step from tokens to clipped gradients and a sampling step, against the
formulas in 64 bits; captured and replayed, on several streams and threads, on
both ways of a Python call, with workspaces of their own and of the caller's."""
import threading

import pytest
import torch

import ends_ref as ref
from test_gpu_embedding import BF, DEV, F32, gen, normal

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R
    from row_reduction_norm_gb300 import api


def near(got, want, what):
    """Norm-wise, as in test_gpu_block.py: six operators and products in fp32 of
    at most 300 terms each, each off by at most 300 u of the sizes of its terms,
    and able to raise what came before by the terms' sizes over their sum (under
    2 here): 2 x 6 x 300 x 2^-24 = 2.2e-4."""
    off = float((got.double() - want).norm() / want.norm())
    assert off <= 2.2e-4, f"{what}: {off:.3g} of its norm off"


def test_training_step_from_tokens_to_clipped_gradients():
    n, vocab, width, scale, eps, beta = 90, 300, 128, 8.0, 1e-6, 0.1
    g = gen(41)
    table, head = normal(g, vocab, width, std=0.1), normal(g, width, vocab, std=width ** -0.5)
    w = normal(g, width, std=0.1) + 1
    ids = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    labels = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    labels[:20] = -1                                            # a prompt
    ids[80:] = -1                                               # padding
    x = R.embedding(ids, table, scale)
    y = R.rms_norm(x, w=w, eps=eps)
    logits = y @ head
    r = R.token_logprobs(logits, labels, entropy=True)
    # minimised: -sum of log probabilities - beta sum of entropies
    dlogits = R.token_logprobs_backward(logits, labels, r.stats, torch.full((n,), -1.0, device=DEV), r.entropy,
                                        torch.full((n,), -beta, device=DEV))
    dhead = y.t() @ dlogits
    dx, dw = R.rms_norm_backward(dlogits @ head.t(), x, w, eps=eps)
    dtable = R.embedding_backward(dx, ids, vocab, scale)
    grads = [dtable, dhead, dw]
    raw = [t.clone() for t in grads]
    norm = R.clip_grad_norm(grads, 1.0)

    v = [t.double().requires_grad_() for t in (table, head, w)]
    there = (ids >= 0)[:, None]
    x64 = torch.where(there, v[0][ids.clamp(min=0)] * scale, 0.0)
    y64 = x64 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + eps) * v[2]
    lp = torch.log_softmax(y64 @ v[1], -1)
    entropy = -(lp.exp() * lp).sum(-1)
    picked = torch.where(labels >= 0, lp.gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
    near(r.logprobs, picked.detach(), "log probabilities")
    near(r.entropy, entropy.detach(), "entropy")
    loss = -picked.sum() - beta * entropy.sum()
    want = torch.autograd.grad(loss, v)
    for name, a, b in zip(("table", "head", "w"), raw, want):
        near(a, b, f"gradient of {name}")
    total = float(torch.stack([b.norm() for b in want]).norm())
    assert abs(float(norm) - total) <= 2.2e-4 * total
    for a, b in zip(grads, want):
        near(a, b / total, "clipped")


def test_sampling_step():
    """Alternatives of a masked row are what sorting gives, and their log probabilities those of given tokens."""
    g, rows, vocab = gen(42), 6, 50257
    x = R.embedding(torch.randint(0, 1000, (rows,), device=DEV, generator=g), normal(g, 1000, 256, dtype=BF))
    logits = R.rms_norm(x) @ normal(g, 256, vocab, dtype=BF, std=0.2)
    logits = logits.masked_fill(torch.rand(rows, vocab, device=DEV, generator=g) < 0.4, float("-inf"))
    r = R.token_logprobs(logits, None, temperature=0.7, top=20, entropy=True)
    assert torch.equal(r.top_ids.long(), ref.likeliest(logits, 20))
    for k in (0, 3, 19):
        one = R.token_logprobs(logits, r.top_ids[:, k].contiguous(), temperature=0.7)
        assert torch.equal(one.logprobs, r.top_logprobs[:, k]) and torch.equal(one.stats, r.stats)


class Work:
    """One call of each operator on its own buffers, all given beforehand."""

    def __init__(self, seed, n=3000, vocab=2000, width=200):
        g = gen(seed)
        self.vocab = vocab
        self.ids = torch.randint(-1, vocab, (n,), device=DEV, generator=g)
        self.table = normal(g, vocab, width, dtype=BF)
        self.few = self.ids[:70].contiguous()
        self.dout = normal(g, n, width, dtype=BF)
        self.logits = normal(g, 50, 5000, dtype=BF, std=3.0)
        self.labels = torch.randint(0, 5000, (50,), device=DEV, generator=g)
        self.g, self.h = normal(g, 50), normal(g, 50)
        self.grads = [normal(g, 70001), normal(g, 333, dtype=BF), normal(g, 100000, dtype=BF)]
        self.out = [torch.empty_like(t) for t in self.grads]
        self.held = torch.zeros(vocab, width, device=DEV)

    def run(self, stream=None):
        k = {"stream": stream}
        r = R.token_logprobs(self.logits, self.labels, 0.9, 7, True, **k)
        return [R.embedding(self.ids, self.table, 2.0, **k),
                R.embedding_backward(self.dout, self.ids, self.vocab, 0.5, **k),
                R.embedding_backward(self.dout, self.ids, self.vocab, out=self.held, **k),
                R.embedding_backward(self.dout[:70], self.few, self.vocab, **k), *r,
                R.token_logprobs_backward(self.logits, self.labels, r.stats, self.g, r.entropy, self.h, 0.9, **k),
                R.clip_grad_norm(self.grads, 10.0, out=self.out, **k), *self.out,
                R.grad_norm(self.grads[1:2], **k)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b)) and len(a) == len(b)


def test_captured_and_replayed_on_other_inputs():
    a, b = Work(1), Work(2)
    want = [[t.clone() for t in w.run()] for w in (a, b)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = a.run()
    for _ in range(3):
        graph.replay()
    assert same(got, want[0])
    fields = ("ids", "table", "few", "dout", "logits", "labels", "g", "h")
    for f in fields:
        getattr(a, f).copy_(getattr(b, f))
    for x, y in zip(a.grads, b.grads):
        x.copy_(y)
    graph.replay()
    assert same(got, want[1])
    # two graphs, each with workspaces of its own, replayed in turn without a wait
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        more = b.run()
    for _ in range(5):
        graph.replay()
        other.replay()
    assert same(got, want[1]) and same(more, want[1])


def test_on_a_stream_of_its_own():
    a = Work(3)
    want = [t.clone() for t in a.run()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = a.run(stream=s)
    s.synchronize()
    assert same(got, want)
    with torch.cuda.stream(s):
        got = a.run()
    s.synchronize()
    assert same(got, want)


def test_several_threads_and_streams_at_once():
    works = [Work(10 + i) for i in range(4)]
    want = [[t.clone() for t in w.run()] for w in works]
    torch.cuda.synchronize()
    bad = []

    def go(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = works[i].run()
            s.synchronize()
            if not same(got, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=go, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_both_ways_of_a_python_call(monkeypatch):
    a = Work(5)
    fast = [t.clone() for t in a.run()]
    monkeypatch.setattr(api, "_fast", api._PythonCalls())
    assert same(a.run(), fast)


def test_workspaces_of_the_callers():
    a = Work(6)
    need = R.rmsnorm_embedding_bwd_workspace_bytes(len(a.ids), a.vocab, 200)
    room = torch.full((need + 64,), 77, dtype=torch.uint8, device=DEV)
    d = R.embedding_backward(a.dout, a.ids, a.vocab, workspace=room[:need])
    assert torch.equal(d, R.embedding_backward(a.dout, a.ids, a.vocab)) and bool((room[need:] == 77).all())
    need = R.rmsnorm_grad_norm_workspace_bytes()
    room = torch.full((need + 64,), 77, dtype=torch.uint8, device=DEV)
    n = R.grad_norm(a.grads, workspace=room[:need])
    assert torch.equal(n, R.grad_norm(a.grads)) and bool((room[need:] == 77).all())


def test_behind_work_that_still_runs():
    """Calls in a row, each on what the one before writes (launches overlap)."""
    g, n, vocab, width = gen(7), 4000, 500, 64
    ids = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    table = torch.randint(-3, 4, (vocab, width), device=DEV, generator=g).float()
    want = table.double()
    for _ in range(4):
        x = R.embedding(ids, table)
        table = R.embedding_backward(x, ids, vocab, 2.0 ** -4)
        R.clip_grad_norm([table], 1e30)
        x64 = want[ids]
        want = torch.zeros_like(want).index_put((ids,), x64, accumulate=True) * 2.0 ** -4
    counts = torch.bincount(ids, minlength=vocab)
    bound = 4 * (counts.max() + 2) * ref.U * want.abs()
    ref.assert_within(table, want, bound, "in a row")
    logits = normal(g, 40, 3000)
    labels = torch.randint(0, 3000, (40,), device=DEV, generator=g)
    x = logits.clone()
    for _ in range(5):
        r = R.token_logprobs(x, labels)
        y = R.token_logprobs_backward(x, labels, r.stats, torch.ones(40, device=DEV), out=x.clone())
        s = R.token_logprobs(x, labels)
        assert torch.equal(r.logprobs, s.logprobs)
        x = y * 100


def test_in_place_clip_in_a_captured_step():
    g = gen(8)
    grads = [normal(g, 5000), normal(g, 90000, dtype=BF)]
    kept = [t.clone() for t in grads]
    total = ref.norm(kept)
    graph = torch.cuda.CUDAGraph()
    R.clip_grad_norm([t.clone() for t in grads], 1.0)
    with torch.cuda.graph(graph):
        n = R.clip_grad_norm(grads, 0.5 * total)
    for _ in range(2):
        for t, k in zip(grads, kept):
            t.copy_(k)
        graph.replay()
        assert abs(float(n) - total) <= 8 * ref.U * total
        for t, k in zip(grads, kept):
            ref.assert_within(t, *ref.clipped(k, total, 0.5 * total), "captured")


def test_gradients_added_up_in_a_captured_step():
    """Two batches into one gradient, as in accumulation over batches: sorted and unsorted tokens."""
    g, vocab, width = gen(9), 700, 72
    ids = [torch.randint(-1, vocab, (n,), device=DEV, generator=g) for n in (5000, 40, 20000)]
    dout = [torch.randint(-8, 9, (len(i), width), device=DEV, generator=g).to(BF) for i in ids]
    total = torch.zeros(vocab, width, device=DEV)
    graph = torch.cuda.CUDAGraph()
    R.embedding_backward(dout[2], ids[2], vocab)
    with torch.cuda.graph(graph):
        total.zero_()
        for i, d in zip(ids, dout):
            R.embedding_backward(d, i, vocab, out=total, accumulate=True)
    want = sum(ref.embedding_backward(d, i, vocab, 1.0)[0] for i, d in zip(ids, dout))
    for _ in range(2):
        graph.replay()
        assert torch.equal(total.double(), want)


@pytest.mark.parametrize("n", [2, 24, 25, 200])
def test_a_tensor_is_not_clipped_twice(n):
    grads = [torch.ones(5, device=DEV) for _ in range(n)]
    twice = grads[:-1] + [grads[0]]
    with pytest.raises(R.RmsNormError):
        R.clip_grad_norm(twice, 1.0)
    assert bool((grads[0] == 1).all())
    # read twice, written to two places: fine
    out = [torch.empty_like(t) for t in twice]
    norm = R.clip_grad_norm(twice, 1.0, out=out)
    assert abs(float(norm) - (5 * n) ** 0.5) <= 1e-5 and torch.equal(out[0], out[-1])
    assert abs(float(R.grad_norm(twice)) - (5 * n) ** 0.5) <= 1e-5
    # tensors without elements may share an address
    R.clip_grad_norm([torch.empty(0, device=DEV)] * 30 + grads, 1.0)
