"""Cases of the operators around a transformer block's matrix products: the
Q+K head norm with rotary positions and its gradients, the append of keys and
values to a paged cache with the same norm and rotation, and the residual
dropout with RMSNorm and its gradients; each in a plain form (elementary
torch operations) and as the package's call."""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_LIMIT = 2 * 8192 * 40 * 128 * 2          # bytes a drawn case of the head operators moves at most
_LIMIT_ROWS = 5 * 8192 * 8192 * 2         # and one of the row operators


def _rope(name, op, dtype, tokens, q_heads, k_heads, head_dim, rot, sections, interleaved, norm, bias, far, pos64):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "q_heads": q_heads, "k_heads": k_heads,
            "head_dim": head_dim, "rot": rot, "sections": sections, "interleaved": interleaved, "norm": norm,
            "bias": bias, "far": far, "pos64": pos64}


def _append(name, dtype, cache, lens, news, pad, q_heads, k_heads, head_dim, rot, interleaved, norm, page, heads_first):
    return {"name": name, "op": "append", "dtype": dtype, "cache": cache, "lens": lens, "news": news, "pad": pad,
            "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim, "rot": rot, "interleaved": interleaved,
            "norm": norm, "page": page, "heads_first": heads_first}


def _rows(name, op, dtype, rows, hidden, p, weight, bias, dh):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "hidden": hidden, "p": p, "weight": weight,
            "bias": bias, "dh": dh}


def _ints(v):
    return ",".join(str(i) for i in v)


def listed():
    return [
        # one decode step of 8 sequences, far into a long context
        _rope("rope_decode_8tok", "rope", "bf16", 8, 32, 8, 128, 128, "64", False, True, 0.0, 131072, True),
        # the packed projection of a prefill or training batch
        _rope("rope_8192tok", "rope", "bf16", 8192, 32, 8, 128, 128, "64", False, True, 0.0, 8192, True),
        # video patches: time, height and width positions, a ragged count, heads of 80, full precision
        _rope("rope_video_4099tok", "rope", "f32", 4099, 16, 16, 80, 80, "8,16,16", False, True, 0.0, 512, False),
        # the gradient of the training batch
        _rope("rope_bwd_8192tok", "rope_bwd", "bf16", 8192, 32, 8, 128, 128, "64", False, True, 0.0, 8192, True),
        # a short odd batch, half of each head rotated, neighbouring pairs, zero-centred weights
        _rope("rope_bwd_1023tok", "rope_bwd", "f32", 1023, 12, 12, 64, 32, "16", True, True, 1.0, 2048, True),
        # a decode step of 64 sequences of many lengths, one new token each
        _append("append_decode_64seq", "bf16", "bf16", _ints(37 * i * i % 2039 for i in range(64)), _ints([1] * 64), 0,
                32, 8, 128, 128, False, True, 16, False),
        # prompts of very different lengths into an 8-bit cache kept head by head, one of them a later chunk
        _append("append_prefill_8bit", "bf16", "e4m3", "0,0,1000,0,4096", "4001,17,1,2085,2088", 0,
                32, 8, 128, 128, False, True, 64, True),
        # chunks, empty sequences and padding rows of a captured batch, odd pages, heads of 96 half rotated
        _append("append_chunks_f32", "f32", "f32", "5,0,333,64,0,7", "100,0,3,1,128,61", 27,
                6, 2, 96, 48, True, False, 7, False),
        # the residual stream of a training step
        _rows("dropout_16384x2048", "dropout", "bf16", 16384, 2048, 0.1, True, 0.0, False),
        # a small full-precision model
        _rows("dropout_f32_64x256", "dropout", "f32", 64, 256, 0.25, True, 0.0, False),
        # its gradient on wide rows, with the gradient of the residual stream joined
        _rows("dropout_bwd_8192x8192", "dropout_bwd", "bf16", 8192, 8192, 0.1, True, 0.0, True),
        # rows of an odd width: no 16-byte alignment, no dropout
        _rows("norm_bwd_f32_1023x1001", "dropout_bwd", "f32", 1023, 1001, 0.0, True, 0.0, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    k = rng.choice([1, 2, 4, 8, 8, 12, 16])
    q = min(48, k * rng.choice([1, 2, 3, 4, 7, 8]))
    d = rng.choice([64, 64, 72, 80, 96, 112, 128, 128, 128, 192, 256, 40])
    part = rng.random()
    if part < 0.6:
        rot = d
    elif part < 0.9:
        rot = 2 * int(d * rng.choice([0.25, 0.4, 0.5, 0.75]) / 2)
    else:
        rot = 2 * rng.randint(4, d // 2)
    return q, k, d, rot


def draw(rng):
    kind = rng.choice(["rope", "rope", "rope_bwd", "append", "append", "dropout", "dropout_bwd", "dropout_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    if kind in ("rope", "rope_bwd"):
        q, k, d, rot = _heads(rng)
        most = max(1, _LIMIT // ((2 if kind == "rope" else 3) * (q + k) * d * size))
        axes = rng.choice([1, 1, 2, 3])
        cuts = sorted(rng.sample(range(1, rot // 2), axes - 1)) if axes > 1 else []
        ends = [0] + cuts + [rot // 2]
        norm = rng.random() < 0.8
        c = _rope("", kind, dtype, _log(rng, 1, min(8192, most)), q, k, d, rot,
                  _ints(b - a for a, b in zip(ends, ends[1:])), rng.random() < 0.4, norm,
                  1.0 if norm and rng.random() < 0.3 else 0.0, rng.choice([512, 8192, 131072, 1 << 20]),
                  rng.random() < 0.5)
    elif kind == "append":
        q, k, d, rot = _heads(rng)
        most = min(8192, _LIMIT // (2 * (q + 2 * k) * d * size))
        seqs = _log(rng, 1, 256)
        if rng.random() < 0.4:
            news = [1] * seqs
        else:
            news = [0 if rng.random() < 0.1 else _log(rng, 1, max(1, min(4096, most // seqs))) for _ in range(seqs)]
            news[rng.randrange(seqs)] += 1
        room = max(1, min(4096, _LIMIT // (4 * k * d * size * seqs)))
        lens = [0 if rng.random() < 0.2 else _log(rng, 1, room) for _ in range(seqs)]
        c = _append("", dtype, rng.choice([dtype, "e4m3"]), _ints(lens), _ints(news), rng.choice([0, 0, 1, 13]), q, k, d,
                    rot, rng.random() < 0.4, rng.random() < 0.8, rng.choice([1, 7, 16, 16, 32, 64, 128]),
                    rng.random() < 0.4)
    else:
        hidden = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            hidden = max(64, hidden // 64 * 64)
        most = max(1, _LIMIT_ROWS // (5 * hidden * size))
        weight = rng.random() < 0.8
        c = _rows("", kind, dtype, _log(rng, 1, min(65536, most)), hidden, rng.choice([0.0, 0.05, 0.1, 0.25, 0.5])
                  if kind == "dropout_bwd" else rng.choice([0.05, 0.1, 0.25, 0.5]), weight,
                  1.0 if weight and rng.random() < 0.3 else 0.0, kind == "dropout_bwd" and rng.random() < 0.6)
    del c["name"]
    return c


def _list(text):
    return [int(v) for v in text.split(",")]


def _inv_freq(rot, base=500000.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (base ** (-2.0 * i / rot)).to(torch.float32)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = _T[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=t):
        return torch.empty(shape, device=dev, dtype=torch.float32).normal_(mean, std, generator=g).to(dtype)

    s = {"case": case, "eps": 1e-6}
    if case["op"] in ("rope", "rope_bwd"):
        n, q, k, d = case["tokens"], case["q_heads"], case["k_heads"], case["head_dim"]
        s["sections"] = _list(case["sections"])
        s["qkv"] = normal(n, (q + 2 * k) * d)            # query, key and value heads of a fused projection
        at = torch.int64 if case["pos64"] else torch.int32
        s["positions"] = torch.randint(0, case["far"], (len(s["sections"]), n), device=dev, generator=g).to(at)
        s["inv_freq"] = _inv_freq(case["rot"]).to(dev)
        s["axis"] = torch.tensor([a for a, m in enumerate(s["sections"]) for _ in range(m)], device=dev)   # of each pair
        centre = 1.0 - case["bias"]
        s["q_w"] = normal(d, std=0.1, mean=centre) if case["norm"] else None
        s["k_w"] = normal(d, std=0.1, mean=centre) if case["norm"] else None
        s["out"] = torch.zeros(n, (q + k) * d, device=dev, dtype=t)
        if case["op"] == "rope_bwd":
            s["dout"] = normal(n, (q + k) * d)
    elif case["op"] == "append":
        q, k, d, page = case["q_heads"], case["k_heads"], case["head_dim"], case["page"]
        lens, news = _list(case["lens"]), _list(case["news"])
        need = [-(-(a + b) // page) for a, b in zip(lens, news)]
        pages, wide = sum(need) + 3, max(max(need), 1) + 1
        order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
        table = torch.full((len(lens), wide), -1, dtype=torch.int32)
        used = 0
        order_host = order.cpu()
        for i, m in enumerate(need):
            table[i, :m] = order_host[used:used + m]
            used += m
        s["total"] = sum(news)
        s["page_table"] = table.to(dev)
        s["cu_tokens"] = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device=dev)
        s["cache_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["qkv"] = normal(s["total"] + case["pad"], (q + 2 * k) * d)
        s["inv_freq"] = _inv_freq(case["rot"]).to(dev)
        s["axis"] = torch.zeros(case["rot"] // 2, dtype=torch.int64, device=dev)
        s["q_w"] = normal(d, std=0.1, mean=1.0) if case["norm"] else None
        s["k_w"] = normal(d, std=0.1, mean=1.0) if case["norm"] else None
        s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if case["cache"] == "e4m3" else (1.0, 1.0)
        for name in ("k_cache", "v_cache"):
            shape = (pages, k, page, d) if case["heads_first"] else (pages, page, k, d)
            if case["cache"] == "e4m3":    # every code but the two NaNs may stand in the cache
                c = torch.randint(0, 256, shape, device=dev, generator=g, dtype=torch.uint8)
                c = torch.where((c & 127) == 127, c - 1, c).view(torch.float8_e4m3fn)
            else:
                c = normal(*shape, dtype=_T[case["cache"]])
            s[name] = c.permute(0, 2, 1, 3) if case["heads_first"] else c      # [pages, page, heads, head_dim]
        s["q_out"] = torch.zeros(s["total"] + case["pad"], q * d, device=dev, dtype=t)
    else:
        n, m = case["rows"], case["hidden"]
        s["w"] = normal(m, std=0.1, mean=1.0 - case["bias"]) if case["weight"] else None
        s["rng"] = torch.randint(0, 1 << 62, (2,), device=dev, generator=g)     # seed and offset
        if case["op"] == "dropout":
            s["x"], s["residual"] = normal(n, m, std=0.5), normal(n, m)
            s["y"], s["h"] = torch.empty(n, m, device=dev, dtype=t), torch.empty(n, m, device=dev, dtype=t)
        else:
            s["dy"], s["h"] = normal(n, m), normal(n, m, std=1.5)
            s["dh"] = normal(n, m) if case["dh"] else None
            s["dres"] = torch.empty(n, m, device=dev, dtype=t)
            s["dx"] = torch.empty(n, m, device=dev, dtype=t) if case["p"] else None
    return s


# ------------------------------------------------------------- plain forms

def _angles(s, positions):
    """cos and sin [tokens, rot / 2] in 32 bits, of angles formed in 64."""
    a = positions.to(torch.float64)[s["axis"]].t() * s["inv_freq"].to(torch.float64)
    return a.cos().to(torch.float32)[:, None, :], a.sin().to(torch.float32)[:, None, :]


def _turn(v, cos, sin, rot, interleaved):
    """The rotation of [tokens, heads, head_dim] values."""
    if interleaved:
        a, b = v[..., 0:rot:2], v[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = v[..., :rot // 2], v[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, v[..., rot:]), -1)


def _head_norm(v, w, bias, eps, norm):
    if not norm:
        return v
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * (w.float() + bias)


def _plain_rope(s):
    c = s["case"]
    q, k, d = c["q_heads"], c["k_heads"], c["head_dim"]
    cos, sin = _angles(s, s["positions"])
    v = s["qkv"][:, :(q + k) * d].float().view(-1, q + k, d)
    n = torch.cat((_head_norm(v[:, :q], s["q_w"], c["bias"], s["eps"], c["norm"]),
                   _head_norm(v[:, q:], s["k_w"], c["bias"], s["eps"], c["norm"])), 1)
    return _turn(n, cos, sin, c["rot"], c["interleaved"]).flatten(1).to(s["qkv"].dtype)


def _head_norm_bwd(g, x, w, bias, eps):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    dw = (g * x * r).sum((0, 1))
    dn = g * (w.float() + bias)
    return r * (dn - x * (r * r * (dn * x).mean(-1, keepdim=True))), dw


def _plain_rope_bwd(s):
    c = s["case"]
    q, k, d = c["q_heads"], c["k_heads"], c["head_dim"]
    t = s["qkv"].dtype
    cos, sin = _angles(s, s["positions"])
    g = _turn(s["dout"].float().view(-1, q + k, d), cos, -sin, c["rot"], c["interleaved"])
    if not c["norm"]:
        return [g.flatten(1).to(t)]
    x = s["qkv"][:, :(q + k) * d].float().view(-1, q + k, d)
    dq, dq_w = _head_norm_bwd(g[:, :q], x[:, :q], s["q_w"], c["bias"], s["eps"])
    dk, dk_w = _head_norm_bwd(g[:, q:], x[:, q:], s["k_w"], c["bias"], s["eps"])
    return [torch.cat((dq, dk), 1).flatten(1).to(t), dq_w.to(t), dk_w.to(t)]


def _plain_append(s):
    c = s["case"]
    q, k, d, page, n = c["q_heads"], c["k_heads"], c["head_dim"], c["page"], s["total"]
    token = torch.arange(n, device=s["qkv"].device)
    seq = (token[:, None] >= s["cu_tokens"][None, 1:]).sum(1)
    at = s["cache_lens"].long()[seq] + token - s["cu_tokens"].long()[seq]
    where, row = s["page_table"].long()[seq, at // page], at % page
    cos, sin = _angles(s, at[None])
    v = s["qkv"][:n].float().view(n, q + 2 * k, d)
    qs = _turn(_head_norm(v[:, :q], s["q_w"], 0.0, s["eps"], c["norm"]), cos, sin, c["rot"], c["interleaved"])
    ks = _turn(_head_norm(v[:, q:q + k], s["k_w"], 0.0, s["eps"], c["norm"]), cos, sin, c["rot"], c["interleaved"])
    s["q_out"][:n] = qs.flatten(1).to(s["q_out"].dtype)
    for cache, new, scale in ((s["k_cache"], ks, s["k_scale"]), (s["v_cache"], v[:, q + k:], s["v_scale"])):
        if c["cache"] == "e4m3":
            codes = (new / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[where, row] = codes.view(torch.uint8)
        else:
            cache[where, row] = new.to(cache.dtype)
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _mul32(a, m):
    """High and low word of the 64-bit product of 32-bit values held in int64."""
    low = (a & 0xFFFF) * m
    high = (a >> 16) * m + (low >> 16)
    return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _kept(case, rng):
    """Which elements dropout keeps: Philox4x32-10, eight 16-bit numbers a block of 8 elements of a row."""
    n, m = case["rows"], case["hidden"]
    blocks = -(-m // 8)
    b = torch.arange(n * blocks, device=rng.device)
    seed, offset = rng[0], rng[1]
    word = torch.zeros_like(b)
    c0, c1, c2, c3 = b & 0xFFFFFFFF, b >> 32, word + (offset & 0xFFFFFFFF), word + (offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    u = torch.stack((c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16), -1)
    return u.view(n, blocks * 8)[:, :m] >= _threshold(case)


def _threshold(case):
    return int(math.floor(case["p"] * 65536.0 + 0.5))


def _plain_dropout(s):
    c = s["case"]
    x = torch.where(_kept(c, s["rng"]), s["x"].float() * (65536.0 / (65536 - _threshold(c))), 0.0)
    h = (s["residual"].float() + x).to(s["x"].dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"])
    if s["w"] is not None:
        y = y * (s["w"].float() + c["bias"])
    return [y.to(h.dtype), h]


def _plain_dropout_bwd(s):
    c = s["case"]
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"])
    g = dy if s["w"] is None else dy * (s["w"].float() + c["bias"])
    d = r * (g - h * (r * r * (g * h).mean(-1, keepdim=True)))
    if s["dh"] is not None:
        d = d + s["dh"].float()
    t = s["h"].dtype
    out = [d.to(t)]
    if c["p"]:
        out.append(torch.where(_kept(c, s["rng"]), d * (65536.0 / (65536 - _threshold(c))), 0.0).to(t))
    if s["w"] is not None:
        out.append((dy * h * r).sum(0).to(t))
    return out


# ------------------------------------------------------- the package's calls

def _own_run(s):
    import row_reduction_norm_gb300 as R
    c = s["case"]
    op = c["op"]
    if op == "rope":
        return R.qk_norm_rope(s["qkv"], c["q_heads"], c["k_heads"], c["head_dim"], s["positions"], s["inv_freq"],
                              q_w=s["q_w"], k_w=s["k_w"], eps=s["eps"], weight_bias=c["bias"], norm=c["norm"],
                              sections=s["sections"], interleaved=c["interleaved"], out=s["out"])
    if op == "rope_bwd":
        dx, dq_w, dk_w = R.qk_norm_rope_backward(
            s["dout"], s["qkv"], c["q_heads"], c["k_heads"], c["head_dim"], s["positions"], s["inv_freq"],
            q_w=s["q_w"], k_w=s["k_w"], eps=s["eps"], weight_bias=c["bias"], norm=c["norm"], sections=s["sections"],
            interleaved=c["interleaved"], out=s["out"])
        return [dx, dq_w, dk_w] if c["norm"] else [dx]
    if op == "append":
        R.qkv_append(s["qkv"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_tokens"], s["cache_lens"],
                     c["q_heads"], c["k_heads"], c["head_dim"], s["inv_freq"], q_w=s["q_w"], k_w=s["k_w"], eps=s["eps"],
                     norm=c["norm"], interleaved=c["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                     q_out=s["q_out"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if op == "dropout":
        return list(R.rms_norm_dropout(s["x"], s["residual"], c["p"], s["rng"], w=s["w"], eps=s["eps"],
                                       weight_bias=c["bias"], out=s["y"], residual_out=s["h"]))
    if not c["p"]:
        d, dw = R.rms_norm_backward(s["dy"], s["h"], w=s["w"], dresidual_out=s["dh"], eps=s["eps"],
                                    weight_bias=c["bias"], out=s["dres"])
        return [d] if dw is None else [d, dw]
    d, dx, dw = R.rms_norm_dropout_backward(s["dy"], s["h"], c["p"], s["rng"], w=s["w"], dresidual_out=s["dh"],
                                            eps=s["eps"], weight_bias=c["bias"], dresidual=s["dres"], dx=s["dx"])
    return [d, dx] if dw is None else [d, dx, dw]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "rope_bwd":
        return _plain_rope_bwd(state)
    if op == "append":
        return _plain_append(state)
    if op == "dropout":
        return _plain_dropout(state)
    return _plain_dropout_bwd(state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("rope", "rope_bwd"):
        values = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        places = case["tokens"] * len(_list(case["sections"])) * (8 if case["pos64"] else 4)
        if case["op"] == "rope":
            return {"bytes": 2 * values * size + places, "flops": 10 * values}
        return {"bytes": (3 if case["norm"] else 2) * values * size + places, "flops": 16 * values}
    if case["op"] == "append":
        n, held = sum(_list(case["news"])), 1 if case["cache"] == "e4m3" else size
        q, k = n * case["q_heads"] * case["head_dim"], n * case["k_heads"] * case["head_dim"]
        return {"bytes": 2 * q * size + 2 * k * (size + held), "flops": 10 * (q + k)}
    values = case["rows"] * case["hidden"]
    if case["op"] == "dropout":
        return {"bytes": 4 * values * size, "flops": 16 * values}
    return {"bytes": (3 + (1 if case["dh"] else 0) + (1 if case["p"] else 0)) * values * size, "flops": 20 * values}


# ------------------------------------------- the definitions, in 64 bits
# Heads as complex numbers, where a rotation is one product; the random words
# with numpy's unsigned 64-bit products; gradients as projections.

def _exact_heads(x, w, bias, eps, norm):
    x = x.double()
    if norm:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * (w.double() + bias)
    return x


def _exact_phase(sections, positions, inv_freq, sign):
    place = torch.cat([p.double()[:, None].expand(-1, m) for p, m in zip(positions, sections)], 1)
    angle = sign * place * inv_freq.double()[None]
    return torch.polar(torch.ones_like(angle), angle)[:, None]


def _exact_turn(v, phase, rot, interleaved):
    out = v.clone()
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    z = torch.complex(v[..., a].contiguous(), v[..., b].contiguous()) * phase
    out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_kept(case, rng):
    n, m = case["rows"], case["hidden"]
    blocks = (m + 7) // 8
    seed, offset = (int(v) for v in rng.tolist())
    b = np.arange(n * blocks, dtype=np.uint64)
    low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [b & low, b >> shift, np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> shift) ^ c[1] ^ np.uint64(key[0]), q & low, (p >> shift) ^ c[3] ^ np.uint64(key[1]), p & low]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    words = np.stack([v.astype(np.uint32) for v in c], -1)
    u = words.reshape(n, blocks * 4).astype("<u4").view("<u2")[:, :m]
    return torch.from_numpy(u >= np.uint16(_threshold(case))).to(rng.device)


def exact(case, seed):
    s = prepare(case, seed)
    eps = s["eps"]
    if case["op"] in ("rope", "rope_bwd"):
        q, k, d, n = case["q_heads"], case["k_heads"], case["head_dim"], case["tokens"]
        x = s["qkv"][:, :(q + k) * d].reshape(n, q + k, d)
        if case["op"] == "rope":
            phase = _exact_phase(s["sections"], s["positions"], s["inv_freq"], 1.0)
            v = torch.cat((_exact_heads(x[:, :q], s["q_w"], case["bias"], eps, case["norm"]),
                           _exact_heads(x[:, q:], s["k_w"], case["bias"], eps, case["norm"])), 1)
            return _exact_turn(v, phase, case["rot"], case["interleaved"]).reshape(n, -1)
        phase = _exact_phase(s["sections"], s["positions"], s["inv_freq"], -1.0)
        g = _exact_turn(s["dout"].double().reshape(n, q + k, d), phase, case["rot"], case["interleaved"])
        if not case["norm"]:
            return [g.reshape(n, -1)]
        x = x.double()
        size = torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps)
        unit = x / size
        dw = g * unit
        g = torch.cat((g[:, :q] * (s["q_w"].double() + case["bias"]), g[:, q:] * (s["k_w"].double() + case["bias"])), 1)
        dx = (g - unit * ((g * unit).sum(-1, keepdim=True) / d)) / size
        return [dx.reshape(n, -1), dw[:, :q].sum((0, 1)), dw[:, q:].sum((0, 1))]
    if case["op"] == "append":
        q, k, d, page, n = case["q_heads"], case["k_heads"], case["head_dim"], case["page"], s["total"]
        lens, news = _list(case["lens"]), _list(case["news"])
        at = torch.cat([torch.arange(a, a + b) for a, b in zip(lens, news)])
        table = s["page_table"].cpu().long()
        where = torch.cat([table[i][torch.arange(a, a + b) // page] for i, (a, b) in enumerate(zip(lens, news))])
        dev = s["qkv"].device
        slot = (where * page + at % page).to(dev)
        phase = _exact_phase([case["rot"] // 2], at[None].to(dev), s["inv_freq"], 1.0)
        x = s["qkv"][:n].reshape(n, q + 2 * k, d)
        rot, inter = case["rot"], case["interleaved"]
        qs = _exact_turn(_exact_heads(x[:, :q], s["q_w"], 0.0, eps, case["norm"]), phase, rot, inter)
        ks = _exact_turn(_exact_heads(x[:, q:q + k], s["k_w"], 0.0, eps, case["norm"]), phase, rot, inter)
        q_out = s["q_out"].double()
        q_out[:n] = qs.reshape(n, -1)
        out = [q_out]
        for cache, new, scale in ((s["k_cache"], ks, s["k_scale"]), (s["v_cache"], x[:, q + k:].double(), s["v_scale"])):
            held = cache.float().double()
            flat = held.reshape(-1, k, d)
            flat[slot] = (new / scale).clamp(-448.0, 448.0) if case["cache"] == "e4m3" else new
            out.append(flat.reshape(held.shape))
        return out
    kept = _exact_kept(case, s["rng"]) if case["p"] else None
    times = 65536.0 / (65536 - _threshold(case))
    m = case["hidden"]
    w = None if s["w"] is None else s["w"].double() + case["bias"]
    if case["op"] == "dropout":
        total = s["residual"].double() + s["x"].double() * times * kept
        h = total.to(s["x"].dtype).double()          # the norm is taken of the sum rounded to its type
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / m + eps)
        return [y if w is None else y * w, total]
    h, dy = s["h"].double(), s["dy"].double()
    size = torch.sqrt((h * h).sum(-1, keepdim=True) / m + eps)
    unit = h / size
    g = dy if w is None else dy * w
    d = (g - unit * ((g * unit).sum(-1, keepdim=True) / m)) / size
    if s["dh"] is not None:
        d = d + s["dh"].double()
    out = [d]
    if case["p"]:
        out.append(d * times * kept)
    if w is not None:
        out.append((dy * unit).sum(0))
    return out
