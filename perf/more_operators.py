"""Cases of the operators at the two ends of a transformer: the lookup of
token embeddings and its gradient, the log probabilities of tokens with
entropy and the likeliest alternatives and their gradient, and the global norm
of all gradients with clipping; each in a plain form (elementary torch
operations) and as the package's call."""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_LIMIT_EMBED = 1 << 30            # bytes a drawn case of the embedding moves at most
_LIMIT_LOGITS = 1 << 31           # of the log probabilities and their gradient
_LIMIT_GRADS = 3 << 30            # and of the clipping


def _embed(name, dtype, tokens, vocab, width, scale, pad, id64):
    return {"name": name, "op": "embed", "dtype": dtype, "tokens": tokens, "vocab": vocab, "width": width,
            "scale": scale, "pad": pad, "id64": id64}


def _embed_bwd(name, dtype, grad, tokens, vocab, width, scale, pad, id64):
    return {"name": name, "op": "embed_bwd", "dtype": dtype, "grad": grad, "tokens": tokens, "vocab": vocab,
            "width": width, "scale": scale, "pad": pad, "id64": id64}


def _logprobs(name, dtype, rows, vocab, extra, temperature, top, entropy, masked, ignored, id64):
    return {"name": name, "op": "logprobs", "dtype": dtype, "rows": rows, "vocab": vocab, "extra": extra,
            "temperature": temperature, "top": top, "entropy": entropy, "masked": masked, "ignored": ignored,
            "id64": id64}


def _logprobs_bwd(name, dtype, rows, vocab, extra, temperature, entropy, masked, ignored, id64):
    return {"name": name, "op": "logprobs_bwd", "dtype": dtype, "rows": rows, "vocab": vocab, "extra": extra,
            "temperature": temperature, "top": 0, "entropy": entropy, "masked": masked, "ignored": ignored,
            "id64": id64}


def _clip(name, sizes, dtypes, ratio):
    return {"name": name, "op": "clip", "sizes": sizes, "dtypes": dtypes, "ratio": ratio}


def _model(layers, hidden, inner, heads, vocab):
    """Parameters of a transformer of the kind the package's operators make up: sizes and types, norms in full precision."""
    layer = [((heads + 2 * max(1, heads // 4)) * 128 * hidden, "bf16"), (heads * 128 * hidden, "bf16"),
             (2 * inner * hidden, "bf16"), (inner * hidden, "bf16"), (hidden, "f32"), (hidden, "f32"), (128, "f32"),
             (128, "f32")]
    every = layers * layer + [(vocab * hidden, "bf16")]
    return _text(n for n, _ in every), _text(t for _, t in every)


def _text(v):
    return ",".join(str(i) for i in v)


def listed():
    return [
        # one decode step of 8 sequences
        _embed("embed_decode_8tok", "bf16", 8, 131072, 4096, 1.0, 0.0, True),
        # a training batch, rows scaled by the root of their width, padding among the tokens
        _embed("embed_16384tok", "bf16", 16384, 131072, 4096, 64.0, 0.02, True),
        # its gradient, into the full-precision gradients that training keeps
        _embed_bwd("embed_bwd_16384tok", "bf16", "f32", 16384, 32768, 4096, 64.0, 0.02, True),
        # many tokens of a small model: narrow rows, the common words thousands of times each
        _embed_bwd("embed_bwd_65536tok", "bf16", "bf16", 65536, 50257, 768, 1.0, 0.0, True),
        # a short batch of odd sizes in full precision
        _embed_bwd("embed_bwd_f32_1023tok", "f32", "f32", 1023, 1009, 1001, 1.0, 0.05, False),
        # sampling for 8 sequences: a grammar masks tokens, the 20 likeliest are reported
        _logprobs("logprobs_decode_8rows", "bf16", 8, 131072, 0, 0.7, 20, True, 0.3, 0.0, True),
        # the tokens of a training batch under the model, with the entropy of each place
        _logprobs("logprobs_8192x131072", "bf16", 8192, 131072, 0, 1.0, 0, True, 0.0, 0.25, True),
        # scoring a text in full precision: an odd vocabulary in padded rows, five alternatives
        _logprobs("logprobs_f32_1001x50257", "f32", 1001, 50257, 47, 1.0, 5, False, 0.0, 0.0, False),
        # the gradient of the training batch, prompts left out, entropy rewarded
        _logprobs_bwd("logprobs_bwd_8192x131072", "bf16", 8192, 131072, 0, 1.0, True, 0.0, 0.25, True),
        # that of a short batch over an odd vocabulary in full precision
        _logprobs_bwd("logprobs_bwd_f32_513x50257", "f32", 513, 50257, 0, 1.3, False, 0.0, 0.1, False),
        # a small model in full precision: many small gradients of odd sizes
        _clip("clip_20_small", _text((257 * (i * i % 89) + 13 * i + 1) for i in range(20)), _text(["f32"] * 20), 0.5),
        # three layers of 4096 and a table: matrices in bf16, norms in full precision
        _clip("clip_25_of_0.56e9", *_model(3, 4096, 8192, 32, 32768), 0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _vocab(rng):
    v = _log(rng, 300, 200000)
    return v if rng.random() < 0.4 else max(64, v // 64 * 64)


def _width(rng):
    w = _log(rng, 64, 8192)
    return w if rng.random() < 0.25 else max(64, w // 64 * 64)


def draw(rng):
    kind = rng.choice(["embed", "embed_bwd", "embed_bwd", "logprobs", "logprobs", "logprobs_bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = _SIZE[dtype]
    if kind in ("embed", "embed_bwd"):
        vocab, width = _vocab(rng), _width(rng)
        scale = 1.0 if rng.random() < 0.5 else round(math.sqrt(width), 3)
        pad, id64 = rng.choice([0.0, 0.0, 0.02, 0.3]), rng.random() < 0.6
        grad = "f32" if dtype == "f32" or rng.random() < 0.5 else "bf16"
        if kind == "embed":
            most = _LIMIT_EMBED // (2 * width * size)
            c = _embed("", dtype, _log(rng, 1, min(65536, most)), vocab, width, scale, pad, id64)
        else:
            vocab = min(vocab, _LIMIT_EMBED // 2 // (width * _SIZE[grad]))
            most = _LIMIT_EMBED // 2 // (width * size)
            c = _embed_bwd("", dtype, grad, _log(rng, 1, min(65536, most)), vocab, width, scale, pad, id64)
    elif kind in ("logprobs", "logprobs_bwd"):
        vocab = _vocab(rng)
        extra = rng.choice([0, 0, 0, rng.randint(1, 200)])
        most = _LIMIT_LOGITS // (vocab * size * (1 if kind == "logprobs" else 2))
        temperature = 1.0 if rng.random() < 0.5 else round(rng.uniform(0.3, 1.7), 2)
        masked, ignored = rng.choice([0.0, 0.0, 0.3, 0.95]), rng.choice([0.0, 0.25])
        entropy, id64 = rng.random() < 0.5, rng.random() < 0.6
        if kind == "logprobs":
            top = rng.choice([0, 0, 1, 5, 20, rng.randint(1, 32)])
            rows = _log(rng, 1, min(8192, most if top == 0 else most // 4))
            c = _logprobs("", dtype, rows, vocab, extra, temperature, top, entropy, masked, ignored, id64)
        else:
            c = _logprobs_bwd("", dtype, _log(rng, 1, min(8192, most)), vocab, extra, temperature, entropy, masked,
                              ignored, id64)
    else:
        if rng.random() < 0.5:
            hidden = 128 * _log(rng, 2, 32)
            heads = max(1, hidden // 128)
            sizes, dtypes = _model(rng.randint(1, 4), hidden, 128 * rng.randint(hidden // 64, hidden // 32), heads,
                                   64 * _log(rng, 8, 512))
        else:
            n = rng.randint(1, 60)
            most = _log(rng, 300, 1 << 21)
            sizes = _text(_log(rng, 1, most) for _ in range(n))
            dtypes = _text(rng.choice(["bf16", "f32", dtype]) for _ in range(n))
        c = _clip("", sizes, dtypes, rng.choice([0.1, 0.5, 0.9, 2.0]))
        if work(c)["bytes"] > _LIMIT_GRADS:
            c = _clip("", *_model(1, 1024, 2048, 8, 4096), 0.5)
    del c["name"]
    return c


def _tokens(case, count, vocab, ignored, dev, g):
    """Token ids as text has them: the r-th most common with a share of log((r + 1) / r), common ones anywhere in the
    vocabulary; -1 where a place is padded or left out."""
    u = torch.rand(count, device=dev, generator=g, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp_(0, vocab - 1)
    ids = torch.randperm(vocab, device=dev, generator=g)[rank]
    if ignored:
        ids = torch.where(torch.rand(count, device=dev, generator=g) < ignored, -1, ids)
    return ids.to(torch.int64 if case["id64"] else torch.int32)


def _distinct(tokens, vocab, ignored):
    """Different ids among so many tokens, in the mean."""
    r = np.arange(1, vocab + 1, dtype=np.float64)
    share = np.log1p(1.0 / r) / math.log(vocab + 1)
    return float((-np.expm1(tokens * (1.0 - ignored) * np.log1p(-np.minimum(share, 1.0 - 1e-12)))).sum())


def _values(text):
    return text.split(",")


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, device=dev, dtype=torch.float32).normal_(0.0, std, generator=g).to(dtype)

    s = {"case": case}
    if op == "embed":
        n, v, d, t = case["tokens"], case["vocab"], case["width"], _T[case["dtype"]]
        s["table"], s["ids"] = normal(v, d, std=0.02, dtype=t), _tokens(case, n, v, case["pad"], dev, g)
        s["out"] = torch.empty(n, d, device=dev, dtype=t)
    elif op == "embed_bwd":
        n, v, d = case["tokens"], case["vocab"], case["width"]
        s["dout"] = normal(n, d, std=0.01, dtype=_T[case["dtype"]])
        s["ids"] = _tokens(case, n, v, case["pad"], dev, g)
        s["grad"] = torch.empty(v, d, device=dev, dtype=_T[case["grad"]])
    elif op in ("logprobs", "logprobs_bwd"):
        n, v, t = case["rows"], case["vocab"], _T[case["dtype"]]
        s["ids"] = _tokens(case, n, v, case["ignored"], dev, g)
        x = normal(n, v + case["extra"], std=2.5)
        # in half of the rows the model is all but sure of the token
        sure = torch.rand(n, device=dev, generator=g) * 16.0 * (torch.rand(n, device=dev, generator=g) < 0.5)
        x.scatter_add_(1, s["ids"].long().clamp(min=0)[:, None], sure[:, None])
        if case["masked"]:
            x.masked_fill_(torch.rand(x.shape, device=dev, generator=g) < case["masked"], float("-inf"))
        s["logits"] = x.to(t)[:, :v]
        if op == "logprobs_bwd":
            s["dlogprobs"] = normal(n, std=1.0 / n)
            s["dentropy"] = normal(n, std=0.01 / n) if case["entropy"] else None
            s["stats"], _, s["entropy"] = _statistics(s["logits"], case["temperature"])[:3]
            s["out"] = torch.empty_like(x, dtype=t)[:, :v]
    else:
        kinds = [_T[k] for k in _values(case["dtypes"])]
        s["grads"] = [normal(int(m), std=0.001, dtype=k) for m, k in zip(_values(case["sizes"]), kinds)]
        s["out"] = [torch.empty_like(v) for v in s["grads"]]
        s["max_norm"] = case["ratio"] * 0.001 * math.sqrt(sum(v.numel() for v in s["grads"]))
    return s


# ------------------------------------------------------------- plain forms

def _plain_embed(s):
    ids, v = s["ids"], s["case"]["vocab"]
    there = ((ids >= 0) & (ids < v))[:, None]
    rows = s["table"][ids.long().clamp(0, v - 1)].float() * s["case"]["scale"]
    return [torch.where(there, rows, 0.0).to(s["table"].dtype)]


def _plain_embed_bwd(s):
    ids, v, dout = s["ids"].long(), s["case"]["vocab"], s["dout"]
    row = torch.where((ids >= 0) & (ids < v), ids, v)            # tokens without a row: one behind the last
    total = torch.zeros(v + 1, dout.shape[1], device=dout.device).index_add_(0, row, dout.float())
    return [(total[:v] * s["case"]["scale"]).to(s["grad"].dtype)]


def _statistics(logits, temperature):
    """(largest logit, log of the sum of the exponentials relative to it) [rows, 2], the distances from the largest
    over the temperature, and the entropy."""
    x = logits.float()
    m = x.amax(-1)
    z = (x - torch.where(m == float("-inf"), 0.0, m)[:, None]) / temperature
    e = z.exp()
    total = e.sum(-1)
    log = total.log()
    # no share, no part in it; a row without any has no entropy
    h = log - torch.where(e > 0, e * z, 0.0).sum(-1) / total
    return torch.stack((m, log), -1), z, torch.where(m == float("-inf"), 0.0, h)


def _likeliest(x, count):
    """Ids of the largest logits, ties to the lowest id: by keys that hold both."""
    bits = (x.float() + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits) * (1 << 31) + (
        x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
    return key.topk(count, -1).indices


def _plain_logprobs(s):
    c, ids = s["case"], s["ids"].long()
    stats, z, entropy = _statistics(s["logits"], c["temperature"])
    low = float("-inf")
    there = (ids >= 0) & (ids < c["vocab"])
    at = z.gather(1, ids.clamp(0, c["vocab"] - 1)[:, None])[:, 0] - stats[:, 1]
    out = [torch.where(there, torch.where(stats[:, 0] == low, low, at), 0.0), stats]
    if c["entropy"]:
        out.append(entropy)
    if c["top"]:
        best = _likeliest(s["logits"], c["top"])
        out += [torch.where(stats[:, :1] == low, low, z.gather(1, best) - stats[:, 1:]), best.to(torch.int32)]
    return out


def _plain_logprobs_bwd(s):
    c, ids, stats = s["case"], s["ids"].long(), s["stats"]
    m = torch.where(stats[:, :1] == float("-inf"), 0.0, stats[:, :1])
    log = (s["logits"].float() - m) / c["temperature"] - stats[:, 1:]
    p = log.exp()
    there = (ids >= 0) & (ids < c["vocab"])
    g = torch.where(there, s["dlogprobs"], 0.0)
    d = -g[:, None] * p
    d.scatter_add_(1, ids.clamp(0, c["vocab"] - 1)[:, None], g[:, None])
    if c["entropy"]:
        d = d - s["dentropy"][:, None] * torch.where(p > 0, p * (log + s["entropy"][:, None]), 0.0)
    d = torch.where(stats[:, :1] == float("-inf"), 0.0, d / c["temperature"])
    return [d.to(s["logits"].dtype)]


def _plain_clip(s):
    squares = torch.stack([v.float().square().sum(dtype=torch.float64) for v in s["grads"]])
    norm = squares.sum().sqrt()
    factor = (s["max_norm"] / norm).clamp(max=1.0).float()
    return [norm.float()[None]] + [(v.float() * factor).to(v.dtype) for v in s["grads"]]


# ------------------------------------------------------- the package's calls

def _own_run(s):
    import row_reduction_norm_gb300 as R
    c = s["case"]
    op = c["op"]
    if op == "embed":
        return [R.embedding(s["ids"], s["table"], scale=c["scale"], out=s["out"])]
    if op == "embed_bwd":
        return [R.embedding_backward(s["dout"], s["ids"], c["vocab"], scale=c["scale"], out=s["grad"])]
    if op == "logprobs":
        r = R.token_logprobs(s["logits"], s["ids"], temperature=c["temperature"], top=c["top"], entropy=c["entropy"])
        out = [r.logprobs, r.stats]
        if c["entropy"]:
            out.append(r.entropy)
        if c["top"]:
            out += [r.top_logprobs, r.top_ids]
        return out
    if op == "logprobs_bwd":
        return [R.token_logprobs_backward(s["logits"], s["ids"], s["stats"], s["dlogprobs"],
                                          entropy=s["entropy"] if c["entropy"] else None, dentropy=s["dentropy"],
                                          temperature=c["temperature"], out=s["out"])]
    return [R.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])] + s["out"]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "embed":
        return _plain_embed(state)
    if op == "embed_bwd":
        return _plain_embed_bwd(state)
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "logprobs_bwd":
        return _plain_logprobs_bwd(state)
    return _plain_clip(state)


def work(case):
    op = case["op"]
    if op in ("embed", "embed_bwd"):
        n, d, size = case["tokens"], case["width"], _SIZE[case["dtype"]]
        ids = n * (8 if case["id64"] else 4)
        if op == "embed":
            return {"bytes": (n + _distinct(n, case["vocab"], case["pad"])) * d * size + ids, "flops": n * d}
        return {"bytes": n * (1.0 - case["pad"]) * d * size + case["vocab"] * d * _SIZE[case["grad"]] + ids,
                "flops": n * d}
    if op in ("logprobs", "logprobs_bwd"):
        n, size = case["rows"], _SIZE[case["dtype"]]
        values = n * case["vocab"]
        few = n * ((8 if case["id64"] else 4) + 16 + 8 * case["top"])
        if op == "logprobs":
            return {"bytes": values * size + few, "flops": (6 if case["entropy"] else 4) * values}
        return {"bytes": 2 * values * size + few, "flops": (8 if case["entropy"] else 5) * values}
    sizes = [(int(m), _SIZE[k]) for m, k in zip(_values(case["sizes"]), _values(case["dtypes"]))]
    return {"bytes": 2 * sum(m * k for m, k in sizes), "flops": 3 * sum(m for m, _ in sizes)}


# ------------------------------------------- the definitions, in 64 bits
# Lookups as rows chosen from a table with one of zeros before it; sums of
# sorted tokens as differences of running totals; log probabilities from torch's
# own log of sums, a block of rows at a time; the norm as one of norms.

def _blocks(n, values):
    step = max(1, (1 << 27) // values)
    return [slice(a, min(n, a + step)) for a in range(0, n, step)]


def _exact_embed(s):
    c = s["case"]
    table = torch.cat((torch.zeros_like(s["table"][:1]), s["table"]))
    ids = s["ids"].long() + 1
    ids[(ids < 1) | (ids > c["vocab"])] = 0
    return [table[ids].double() * c["scale"]]


def _exact_embed_bwd(s):
    c, ids = s["case"], s["ids"].long()
    order = torch.argsort(ids, stable=True)
    held = ids[order]
    row = torch.arange(c["vocab"], device=ids.device)
    first, last = torch.searchsorted(held, row), torch.searchsorted(held, row, right=True)

    def columns(a):
        run = s["dout"][:, a:a + 512][order].double().cumsum(0)
        run = torch.cat((torch.zeros_like(run[:1]), run))
        return (run[last] - run[first]) * c["scale"]

    return [torch.cat([columns(a) for a in range(0, c["width"], 512)], 1)]


def _exact_logprobs(s):
    c = s["case"]
    low = float("-inf")

    def block(rows):
        x, ids = s["logits"][rows].double(), s["ids"][rows].long()
        m = x.max(-1, keepdim=True).values
        none = m == low
        shifted = torch.nan_to_num(x - m, nan=low, neginf=low) / c["temperature"]
        log = torch.logsumexp(shifted, -1, keepdim=True)
        lp = torch.where(none, low, shifted - log)
        there = (ids >= 0) & (ids < c["vocab"])
        got = [torch.where(there, lp.gather(1, ids.clamp(0, c["vocab"] - 1)[:, None])[:, 0], 0.0),
               torch.cat((m, log), 1)]
        if c["entropy"]:
            got.append(torch.special.entr(lp.exp()).sum(-1))
        if c["top"]:
            best = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
            got += [lp.gather(1, best), best.to(torch.int32)]
        return got

    return [torch.cat(v) for v in zip(*[block(rows) for rows in _blocks(c["rows"], c["vocab"])])]


def _exact_logprobs_bwd(s):
    c = s["case"]

    def block(rows):
        x, ids = s["logits"][rows].double() / c["temperature"], s["ids"][rows].long()
        none = x.amax(-1, keepdim=True) == float("-inf")
        p = torch.where(none, 0.0, torch.softmax(torch.where(none, 0.0, x), -1))
        there = (ids >= 0) & (ids < c["vocab"]) & ~none[:, 0]
        onto = torch.zeros_like(p)
        onto[there.nonzero()[:, 0], ids[there]] = 1.0
        d = s["dlogprobs"][rows].double()[:, None] * (onto - p) * there[:, None]
        if c["entropy"]:
            surprise = torch.special.entr(p)                     # -p log p
            d += s["dentropy"][rows].double()[:, None] * (surprise - p * surprise.sum(-1, keepdim=True))
        return d / c["temperature"]

    return [torch.cat([block(rows) for rows in _blocks(c["rows"], c["vocab"])])]


def _exact_clip(s):
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(v.double()) for v in s["grads"]]))
    factor = min(1.0, s["max_norm"] / float(norm))
    return [norm[None]] + [v.double() * factor for v in s["grads"]]


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"embed": _exact_embed, "embed_bwd": _exact_embed_bwd, "logprobs": _exact_logprobs,
                "logprobs_bwd": _exact_logprobs_bwd, "clip": _exact_clip}[case["op"]](s)
