"""What is measured of a quantized decoder layer's further operators: the gradient of a product with the
sweep's codes (gptq_linear_backward), the gated feed-forward block on two members' codes and its
gradient (gptq_gated, gptq_gated_backward), rotary positions (gptq_rotary), and the eviction of cached
tokens by the attention they have received (gptq_cache_score, gptq_cache_evict).

``run`` computes a case in plain torch operations (``own`` false) or with the framework's calls
(``own`` true), from the same state.  ``exact`` is the definition in 64 bits.

Codes of a weight matrix are the sweeps' planes: q4tp keeps column 2m in the low nibble of byte m
and 2m + 1 in the high one, value (q - 8) s; q2tp keeps column 4m + i in bits 2i of byte m, value
(q - 1.5) s; s is f32, one per row and 32 columns.

A key's row of the 4-bit cache holds, with G = D / 32, word (h, g) of 4 bytes at 4 (h G + g), h < 4:
nibble k of it is channel 32 g + 8 h + 2 k, nibble k + 4 the channel after; the nibble is c + 8, the
value c s, s one bf16 per token, head and 32 channels ([pages, heads, page, G]).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _import():
    import post_weight_quantization_amd as pwq
    return pwq


# ---------------------------------------------------------------------------------- the cases

def listed():
    gated = {"op": "gated", "codec": "q4tp", "act": "silu", "bias": False}
    grad = {**gated, "op": "gated_grad"}
    rotary = {"op": "rotary", "q_heads": 32, "heads": 8, "dim": 128, "part": 128, "far": 4096, "stretch": 1.0, "backward": False}
    cache = {"heads": 8, "dim": 128, "page": 16}
    return [
        # A few odd tokens' gradient through a 2-bit calibration layer, in f32.
        {"name": "linear_grad_calibration", "op": "linear_grad", "t": 37, "rows": 2048, "n": 8192, "codec": "q2tp", "type": "f32"},
        # A whole prompt's gradient through the 17408-wide down projection.
        {"name": "linear_grad_prompt", "op": "linear_grad", "t": 4096, "rows": 5120, "n": 17408, "codec": "q4tp", "type": "bf16"},
        # One token through a middling feed-forward block: latency.
        {"name": "gated_one_token", **gated, "t": 1, "rows": 8192, "n": 2048, "type": "bf16"},
        # A whole prompt through the block of the 5120-wide layer: the largest product.
        {"name": "gated_prompt_4096", **gated, "t": 4096, "rows": 17408, "n": 5120, "type": "bf16"},
        # The tuning of a small layer on one odd short sequence, with biases.
        {"name": "gated_grad_small", **grad, "t": 333, "rows": 4096, "n": 2048, "type": "f32", "act": "gelu", "bias": True},
        # A training step's sequences through the block of the 5120-wide layer.
        {"name": "gated_grad_2000", **grad, "t": 2000, "rows": 17408, "n": 5120, "type": "f16"},
        # One new token of each of 48 sequences.
        {"name": "rotary_decode_48", **rotary, "rows": 48, "layout": "half", "type": "bf16"},
        # Long prompts, half of each head rotated, neighbours paired, positions stretched to a long context.
        {"name": "rotary_prompts", **rotary, "rows": 20000, "layout": "interleaved", "part": 64, "far": 131072, "stretch": 8.0,
         "type": "f16"},
        # What the single rows of a serving batch have paid attention to.
        {"name": "score_decode_64", "op": "score", **cache, "seqs": 64, "rows": 1, "len": 4096, "group": 8, "type": "bf16",
         "window": 0, "sinks": 0},
        # The same of chunks of prompts, over what is cached already.
        {"name": "score_prompt_chunk", "op": "score", **cache, "seqs": 2, "rows": 1000, "len": 8192, "group": 4, "heads": 4,
         "type": "bf16", "window": 0, "sinks": 0},
        # One user's cache cut back to a budget: latency.
        {"name": "evict_one", "op": "evict", **cache, "seqs": 1, "len": 1500, "keep": 1024, "sinks": 4, "recent": 64},
        # A serving batch's.
        {"name": "evict_batch_32", "op": "evict", **cache, "seqs": 32, "len": 8192, "keep": 2048, "sinks": 4, "recent": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_grad", "gated", "gated", "gated_grad", "rotary", "score", "evict"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("linear_grad", "gated", "gated_grad"):
        n, rows, t = 32 * _log(rng, 8, 200), _log(rng, 200, 12000), _log(rng, 1, 4096)
        most = 20000000000 if kind == "f32" else 150000000000
        t = max(1, min(t, most // (n * rows)))
        case = {"op": op, "t": t, "rows": rows, "n": n, "codec": rng.choice(["q4tp", "q4tp", "q2tp"]), "type": kind}
        if op != "linear_grad":
            case.update(act=rng.choice(["none", "relu", "silu", "silu", "gelu", "gelu_tanh"]), bias=rng.random() < 0.4)
        return case
    if op == "rotary":
        dim = rng.choice([64, 80, 96, 128, 256])
        return {"op": op, "rows": _log(rng, 1, 20000), "q_heads": rng.choice([1, 4, 7, 16, 32]), "heads": rng.choice([1, 2, 4, 8]),
                "dim": dim, "part": dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2), "far": _log(rng, 2000, 1000000),
                "stretch": rng.choice([1.0, 1.0, 4.0, 16.0]), "layout": rng.choice(["half", "interleaved"]),
                "backward": rng.random() < 0.3, "type": kind}
    case = {"op": op, "heads": rng.randint(1, 12), "dim": rng.choice([64, 128, 256]), "page": rng.choice([16, 32, 64, 128])}
    if op == "evict":
        seqs = _log(rng, 1, 32)
        length = _log(rng, 40, 8192)
        keep = _log(rng, 20, length)
        sinks = rng.choice([0, 1, 4])
        return {**case, "seqs": seqs, "len": length, "keep": keep, "sinks": sinks, "recent": rng.randint(0, (keep - sinks) // 2)}
    if rng.random() < 0.6:
        rows, seqs = rng.choice([1, 1, 1, 2, 5]), _log(rng, 1, 48)
        group, length = rng.choice([1, 2, 3, 4, 7, 8, 16]), _log(rng, 16, 4096 if seqs > 12 else 12000)
    else:
        rows, seqs, group = _log(rng, 16, 1000), rng.randint(1, 3), rng.choice([1, 2, 4, 5, 8])
        length = rows + _log(rng, 1, 3500)
        case["heads"] = rng.randint(1, 4)
    window = 0 if rng.random() < 0.6 else _log(rng, 8, 2000)
    return {**case, "seqs": seqs, "rows": rows, "len": max(length, rows), "group": group, "type": kind, "window": window,
            "sinks": rng.choice([0, 1, 4, 64]) if window else 0}


# ---------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 41)


def _weights(g, rows, n, codec):
    """Codes and scales of one quantized matrix, as a sweep returns them: rungs of a ladder."""
    if codec == "q4tp":
        q = (torch.randn(rows, n, device="cuda", generator=g) * 2.9).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
        codes = q[:, 0::2] | (q[:, 1::2] << 4)
    else:
        q = torch.randint(0, 4, (rows, n), device="cuda", generator=g, dtype=torch.uint8)
        codes = q[:, 0::4] | (q[:, 1::4] << 2) | (q[:, 2::4] << 4) | (q[:, 3::4] << 6)
    lo = -8.5 + torch.rand(rows, 1, device="cuda", generator=g)
    c = torch.randint(0, 32, (rows, n // 32), device="cuda", generator=g)
    return codes, torch.exp2(lo + c * 0.06)


def _lengths(case):
    """Cached tokens of each sequence, and how many of them are rows of this call: sizes, so the case's alone."""
    B, L, R = case["seqs"], case["len"], case.get("rows", 1)
    r = np.random.RandomState(29 * B + 13 * R + L)
    rows = np.full(B, R) if R <= 8 else np.maximum(1, np.round(R * r.uniform(0.5, 1.0, B))).astype(int)
    n = np.maximum(rows, np.round(L * r.uniform(0.4, 1.0, B)).astype(int))
    n[r.randint(B)] = L
    return n, rows


def _tables(case, seed, wanted):
    """Pages in an order without pattern: one table for each list of token counts in `wanted`, and how many pages."""
    r = np.random.RandomState((int(seed) * 137 + 11) % (1 << 31))
    blocks = [-(-np.asarray(w) // case["page"]) for w in wanted]
    total = int(sum(b.sum() for b in blocks))
    pages, tables = r.permutation(total + 3)[:total].astype(np.int32), []
    for b in blocks:
        table = np.zeros((len(b), int(b.max())), np.int32)
        table[np.arange(table.shape[1])[None, :] < b[:, None]] = pages[: int(b.sum())]
        pages = pages[int(b.sum()):]
        tables.append(torch.from_numpy(table).cuda())
    return tables, total + 3


def _key_codes(case, seed, pages):
    """Codes 1..15 of a whole cache's keys, channels in order, and their scales."""
    g = _gen(seed + 2)
    shape = (pages, case["heads"], case["page"], case["dim"])
    q = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, 2.9, generator=g)
    q = (q.round_().clamp_(-7, 7) + 8).to(torch.uint8)
    z = torch.empty(shape[:3] + (case["dim"] // 32,), dtype=torch.float32, device="cuda").normal_(0.0, 0.3, generator=g)
    s = (z.exp() * 0.35).view(torch.int32) & ~0x7FFFF  # 5 significant bits
    return q, s.view(torch.float32).to(torch.bfloat16)


def _pack_keys(q):
    """[..., D] codes in order -> [..., D / 2] bytes of key rows."""
    G = q.shape[-1] // 32
    x = q.view(*q.shape[:-1], G, 4, 4, 2)                       # g, h, k, parity
    x = x.movedim(-4, -3)                                       # h, g, k, parity
    x = torch.cat([x[..., 0], x[..., 1]], -1)                   # h, g, 8 nibbles
    return (x[..., 0::2] | (x[..., 1::2] << 4)).reshape(*q.shape[:-1], G * 16)


def _frequencies(case):
    """Of each pair of channels, with the angles of long contexts stretched: pairs that turn often keep theirs, slow
    ones are slowed down, and a ramp lies between."""
    half = case["part"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    if case["stretch"] != 1.0:
        turns = 4096.0 * f / (2.0 * math.pi)
        ramp = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * ramp + f / case["stretch"] * (1.0 - ramp)
    return f


def _factor(case):
    return 1.0 if case["stretch"] == 1.0 else 0.1 * math.log(case["stretch"]) + 1.0


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    st = {"case": case}
    if op in ("linear_grad", "gated", "gated_grad"):
        kind, t, rows, n = TYPES[case["type"]], case["t"], case["rows"], case["n"]
        st["gate"] = _weights(g, rows, n, case["codec"])
        if op != "linear_grad":
            st["up"] = _weights(g, rows, n, case["codec"])
            # Activations with a few loud channels, as the calibration workloads have.
            loud = torch.where(torch.rand(n, device="cuda", generator=g) < 0.01, 8.0, 1.0)
            st["x"] = (torch.randn(t, n, device="cuda", generator=g) * loud).to(kind)
            st["bias"] = [torch.randn(rows, device="cuda", generator=g) * 0.5 if case["bias"] else None for _ in range(2)]
        if op != "gated":
            # Gradients of a mean over some hundred tokens: small, tokens unlike each other.
            size = torch.exp2(torch.randn(t, 1, device="cuda", generator=g) - 8.0)
            st["dy"] = (torch.randn(t, rows, device="cuda", generator=g) * size).to(kind)
        return st
    if op == "rotary":
        rows, hq, hk, dim = case["rows"], case["q_heads"], case["heads"], case["dim"]
        x = torch.randn(rows, hq + 2 * hk, dim, device="cuda", generator=g).to(TYPES[case["type"]])
        st["q"], st["k"], _ = x.split([hq, hk, hk], 1)  # slices of one projection's output
        st["position"] = torch.randint(0, case["far"], (rows,), device="cuda", generator=g, dtype=torch.int32)
        if rows > 64:  # a prompt's rows in their order
            st["position"] = st["position"][:1] + torch.arange(rows, device="cuda", dtype=torch.int32)
        st["freq"], st["factor"] = _frequencies(case), _factor(case)
        return st
    length, rows = _lengths(case)
    st["length"] = torch.from_numpy(length.astype(np.int32)).cuda()
    st["width"] = int(length.max())
    if op == "evict":
        (st["table"], st["into"]), pages = _tables(case, seed, [length, np.minimum(length, case["keep"])])
        shape = (pages, case["heads"], case["page"])
        st["cache"] = [torch.randint(0, 256, shape + (case["dim"] // 2,), device="cuda", generator=g, dtype=torch.uint8) for _ in range(2)]
        st["cache"] += [(torch.randn(*shape, case["dim"] // 32, device="cuda", generator=g) * 0.3).exp().to(torch.bfloat16) for _ in range(2)]
        # Sums of softmax weights: many near nothing, a few heavy ones, and many that no row has looked at.
        z = torch.exp(2.0 * torch.randn(shape, device="cuda", generator=g) - 6.0)
        st["score"] = torch.where(torch.rand(shape, device="cuda", generator=g) < 0.1, 0.0, z)
        return st
    (st["table"],), pages = _tables(case, seed, [length])
    start = np.concatenate([[0], np.cumsum(rows)])
    st["rows"], st["most"], st["single"] = int(start[-1]), int(rows.max()), bool((rows == 1).all())
    st["start"] = torch.from_numpy(start.astype(np.int32)).cuda()
    codes, scales = _key_codes(case, seed, pages)
    keys = _pack_keys(codes)
    st["cache"] = (keys, torch.full_like(keys, 0x88), scales, torch.ones_like(scales))  # the values are not looked at
    shape = (pages, case["heads"], case["page"])
    st["q"] = _queries(case, seed, st["rows"])
    st["score"] = _old_score(case, seed, shape)
    st["out"] = torch.zeros(shape, device="cuda")
    w = _plain_logits(st)
    lse = torch.logsumexp(w, -1)                                          # [B, H, group, R]
    st["lse"] = _packed_rows(st, lse.permute(0, 3, 1, 2).flatten(2)).contiguous()
    return st


def _queries(case, seed, total):
    g = _gen(seed + 3)
    x = torch.randn(total, case["heads"] * case["group"], case["dim"], device="cuda", generator=g)
    return x.to(TYPES[case["type"]])


def _old_score(case, seed, shape):
    return torch.exp(2.0 * torch.randn(shape, device="cuda", generator=_gen(seed + 4)) - 6.0)


# ---------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear_grad": _own_linear_grad, "gated": _own_gated, "gated_grad": _own_gated_grad, "rotary": _own_rotary,
                "score": _own_score, "evict": _own_evict}[op](state)
    return {"linear_grad": _plain_linear_grad, "gated": _plain_gated, "gated_grad": _plain_gated_grad, "rotary": _plain_rotary,
            "score": _plain_score, "evict": _plain_evict}[op](state)


def _own_linear_grad(s):
    return _import().gptq_linear_backward(s["dy"], *s["gate"], codec=s["case"]["codec"])


def _own_gated(s):
    c = s["case"]
    return _import().gptq_gated(s["x"], s["gate"], s["up"], codec=c["codec"], act=c["act"], gate_bias=s["bias"][0],
                                up_bias=s["bias"][1])


def _own_gated_grad(s):
    c = s["case"]
    return _import().gptq_gated_backward(s["dy"], s["x"], s["gate"], s["up"], codec=c["codec"], act=c["act"],
                                         gate_bias=s["bias"][0], up_bias=s["bias"][1])


def _own_rotary(s):
    c = s["case"]
    return _import().gptq_rotary(s["q"], s["position"], s["freq"], K=s["k"], layout=c["layout"], factor=s["factor"],
                                 backward=c["backward"])


def _own_score(s):
    c = s["case"]
    return _import().gptq_cache_score(s["cache"], s["q"], s["lse"], s["score"], s["table"], s["length"],
                                      start=None if s["single"] else s["start"], window=c["window"], sinks=c["sinks"],
                                      out=s["out"])


def _own_evict(s):
    c = s["case"]
    length, index = _import().gptq_cache_evict(s["cache"], s["table"], s["length"], s["score"], c["keep"], sinks=c["sinks"],
                                               recent=c["recent"], into=s["into"])
    return [length, index, s["score"], *s["cache"]]


def _plain_weights(codes, scale, codec):
    if codec == "q4tp":
        w = torch.stack([codes & 15, codes >> 4], -1).float() - 8.0
    else:
        w = torch.stack([codes & 3, (codes >> 2) & 3, (codes >> 4) & 3, codes >> 6], -1).float() - 1.5
    return (w.view(scale.shape[0], scale.shape[1], 32) * scale[..., None]).flatten(1)


def _plain_act(z, act):
    """The activation and its derivative."""
    if act == "relu":
        return torch.clamp_min(z, 0.0), (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-k * (z + 0.044715 * z * z * z)))
        return z * s, s + z * s * (1.0 - s) * k * (1.0 + 3.0 * 0.044715 * z * z)
    return z, torch.ones_like(z)


def _plain_linear_grad(s):
    w = _plain_weights(*s["gate"], s["case"]["codec"])
    return (s["dy"].float() @ w).to(s["dy"].dtype)


def _plain_sums(s, which, k):
    w = _plain_weights(*s[which], s["case"]["codec"])
    z = s["x"].float() @ w.t()
    return w, z if s["bias"][k] is None else z + s["bias"][k]


def _plain_gated(s):
    _, a = _plain_sums(s, "gate", 0)
    _, b = _plain_sums(s, "up", 1)
    return (_plain_act(a, s["case"]["act"])[0] * b).to(s["x"].dtype)


def _plain_gated_grad(s):
    wg, a = _plain_sums(s, "gate", 0)
    wu, b = _plain_sums(s, "up", 1)
    y, slope = _plain_act(a, s["case"]["act"])
    dy = s["dy"].float()
    return ((dy * b * slope) @ wg + (dy * y) @ wu).to(s["x"].dtype)


def _plain_turned(s, x):
    c = s["case"]
    angle = s["position"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    if c["backward"]:
        sin = -sin
    v, half = x.float(), c["part"] // 2
    if c["layout"] == "half":
        a, b = v[..., :half], v[..., half:c["part"]]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = v[..., 0:c["part"]:2], v[..., 1:c["part"]:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, v[..., c["part"]:]], -1).to(x.dtype)


def _plain_rotary(s):
    return _plain_turned(s, s["q"]), _plain_turned(s, s["k"])


def _packed_rows(s, x):
    """[B, most rows, ...] -> [rows, ...]."""
    i = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["start"][1:], i, right=True)
    return x[b, i - s["start"][b].long()]


def _plain_logits(s):
    """Scores [B, heads, group, rows, tokens], f32, what a row does not see at -inf."""
    c = s["case"]
    B, H, D, R, L, group = c["seqs"], c["heads"], c["dim"], s["most"], s["width"], c["group"]
    rows = s["start"][1:] - s["start"][:-1]
    pos = torch.arange(L, device="cuda")
    at = torch.minimum(pos[None, :], s["length"][:, None] - 1).long()
    p, o = s["table"][torch.arange(B, device="cuda")[:, None], at // c["page"]].long(), at % c["page"]
    w = s["cache"][0][p, :, o].unflatten(-1, (4, D // 32, 4))
    w = torch.stack([w & 15, w >> 4], -1).flatten(-2)                  # h, g, nibble
    w = torch.stack([w[..., :4], w[..., 4:]], -1).flatten(-2)          # h, g, channel
    keys = w.transpose(-2, -3).flatten(-2).float() - 8.0               # g, channel of the group
    keys = (keys * s["cache"][2][p, :, o].float()[..., None]).flatten(-2)                # [B, L, H, D]
    i = torch.arange(R, device="cuda")
    take = torch.minimum(s["start"][:-1, None] + i[None, :], s["start"][1:, None] - 1).long()
    q = s["q"].float()[take].view(B, R, H, group, D).permute(0, 2, 3, 1, 4).reshape(B * H, group * R, D)
    w = torch.bmm(q, keys.permute(0, 2, 3, 1).reshape(B * H, D, L)).mul_(1.0 / math.sqrt(D)).view(B, H, group, R, L)
    at = s["length"][:, None] - rows[:, None] + i[None, :]                               # [B, R]
    seen = (pos <= at[..., None]) & (i[None, :] < rows[:, None])[..., None]
    if c["window"]:
        seen &= (pos > at[..., None] - c["window"]) | (pos < c["sinks"])
    return w.masked_fill_(~seen[:, None, None], -math.inf)


def _plain_score(s):
    c = s["case"]
    w = _plain_logits(s)
    B, L = c["seqs"], s["width"]
    rows = s["start"][1:] - s["start"][:-1]
    take = torch.minimum(s["start"][:-1, None] + torch.arange(s["most"], device="cuda"), s["start"][1:, None] - 1).long()
    lse = s["lse"][take].view(B, s["most"], c["heads"], c["group"]).permute(0, 2, 3, 1)
    paid = torch.exp(w - lse[..., None]).sum((2, 3))                                     # [B, H, L]
    pos = torch.arange(L, device="cuda")
    at = torch.minimum(pos[None, :], s["length"][:, None] - 1)                           # behind the end the last again
    p, o = s["table"][torch.arange(B, device="cuda")[:, None], at // c["page"]].long(), (at % c["page"]).long()
    old = s["score"][p, :, o] * (at < s["length"][:, None] - rows[:, None])[..., None]   # [B, L, H]
    s["out"][p, :, o] = old + paid.gather(2, at.long()[:, None].expand(-1, c["heads"], -1)).transpose(1, 2)
    return s["out"]


def _plain_evict(s):
    c = s["case"]
    B, H, L, keep, page = c["seqs"], c["heads"], s["width"], c["keep"], c["page"]
    n = torch.clamp_max(s["length"], keep)
    pos = torch.arange(L, device="cuda")
    at = torch.minimum(pos[None, :], s["length"][:, None] - 1).long()
    b = torch.arange(B, device="cuda")[:, None]
    z = s["score"][s["table"][b, at // page].long(), :, at % page].transpose(1, 2)       # [B, H, L]
    always = (pos < c["sinks"]) | (pos >= s["length"][:, None] - c["recent"])
    z = torch.where(always[:, None], math.inf, z)
    z = torch.where(pos < s["length"][:, None, None], z, -math.inf)
    order = torch.sort(z, dim=-1, descending=True, stable=True)[1][..., :keep]               # ties: the lowest first
    if L < keep:
        order = torch.nn.functional.pad(order, (0, keep - L), value=L)
    j = torch.arange(keep, device="cuda")
    order = torch.where(j < n[:, None, None], order, L)
    index = torch.sort(order, -1)[0]                                                     # [B, H, keep]
    found = torch.where(j < n[:, None, None], index, -1).to(torch.int32)
    # Places past a sequence's end stand for its last token again.
    last = torch.minimum(j[None, :], n[:, None] - 1).long()                              # [B, keep]
    src = index.gather(2, last[:, None].expand(-1, H, -1))
    h = torch.arange(H, device="cuda")[:, None]
    sp, so = s["table"][b[..., None], src // page].long(), src % page
    dp, do = s["into"][b, last // page].long()[:, None], (last % page)[:, None]
    for plane in (s["score"], *s["cache"]):
        plane[dp, h, do] = plane[sp, h, so]
    return [n, found, s["score"], *s["cache"]]


# ---------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("linear_grad", "gated", "gated_grad"):
        e, t, rows, n = (4 if case["type"] == "f32" else 2), case["t"], case["rows"], case["n"]
        held = rows * n // (2 if case["codec"] == "q4tp" else 4) + rows * (n // 32) * 4
        if op == "linear_grad":
            return {"bytes": held + t * (rows + n) * e, "flops": 2 * t * rows * n}
        held = 2 * held + (8 * rows if case["bias"] else 0)
        if op == "gated":
            return {"bytes": held + t * (rows + n) * e, "flops": 4 * t * rows * n}
        return {"bytes": held + t * (rows + 2 * n) * e, "flops": 8 * t * rows * n}
    if op == "rotary":
        e, heads = (4 if case["type"] == "f32" else 2), case["q_heads"] + case["heads"]
        return {"bytes": case["rows"] * (heads * case["dim"] * 2 * e + 4) + 4 * case["part"],
                "flops": case["rows"] * heads * case["part"] * 3}
    length, rows = _lengths(case)
    H, D = case["heads"], case["dim"]
    if op == "evict":
        kept = np.minimum(length, case["keep"])
        token = H * (D * 2 * 18 // 32 + 4)          # codes, scales and score of a token
        return {"bytes": int(length.sum() * H * 4 + kept.sum() * (2 * token + 4 * H)), "flops": int(length.sum() * H)}
    e, seen, pairs = (4 if case["type"] == "f32" else 2), 0, 0
    for n, r in zip(length.tolist(), rows.tolist()):
        p = np.arange(n - r, n)
        low = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros(r, int)
        pairs += int((p - low + 1 + np.minimum(low, case["sinks"])).sum())
        seen += int(n - low[0] + min(low[0], case["sinks"]))
    q = int(rows.sum()) * H * case["group"]
    return {"bytes": int(seen * H * D * 18 / 32 + 8 * H * length.sum() + q * (D * e + 4)), "flops": 2 * pairs * H * case["group"] * D}


# ---------------------------------------------------------------------------------- the definition, 64 bits

def _exact_weights(codes, scale, codec):
    per = 2 if codec == "q4tp" else 4
    shift = torch.arange(per, device="cuda", dtype=torch.uint8) * (8 // per)
    levels = ((codes[:, :, None] >> shift) & (2 ** (8 // per) - 1)).reshape(codes.shape[0], -1).double()
    return (levels - (8.0 if per == 2 else 1.5)) * scale.double().repeat_interleave(32, 1)


def _exact_gated(x, wg, wu, bias, act):
    a, b = x @ wg.t(), x @ wu.t()
    a, b = (z if k is None else z + k.double() for z, k in ((a, bias[0]), (b, bias[1])))
    if act == "relu":
        a = a * (a > 0)
    elif act == "silu":
        a = a * torch.sigmoid(a)
    elif act == "gelu":
        a = a * torch.special.ndtr(a)
    elif act == "gelu_tanh":
        a = 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)))
    return a * b


def exact(case, seed):
    op = case["op"]
    if op == "evict":
        return None  # nothing is computed: what is kept is moved as it is
    st = prepare(case, seed)
    if op == "linear_grad":
        return st["dy"].double() @ _exact_weights(*st["gate"], case["codec"])
    if op in ("gated", "gated_grad"):
        w = [_exact_weights(*st[k], case["codec"]) for k in ("gate", "up")]
        x = st["x"].double()
        if op == "gated":
            return _exact_gated(x, *w, st["bias"], case["act"])
        x.requires_grad_()
        return torch.autograd.grad(_exact_gated(x, *w, st["bias"], case["act"]), x, st["dy"].double())[0]
    if op == "rotary":
        return [_exact_turned(st, x) for x in (st["q"], st["k"])]
    pages = st["out"].shape[0]
    codes, scales = _key_codes(case, seed, pages)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    length, rows = _lengths(case)
    start = np.concatenate([[0], np.cumsum(rows)])
    for i, (n, r) in enumerate(zip(length.tolist(), rows.tolist())):
        at = torch.arange(n, device="cuda")
        page = st["table"][i, at // case["page"]].long()
        k = (codes[page, :, at % case["page"]].double() - 8.0) * scales[page, :, at % case["page"]].double().repeat_interleave(32, -1)
        x = st["q"][start[i]: start[i] + r].double().unflatten(1, (case["heads"], case["group"]))
        p = torch.arange(n - r, n, device="cuda")[:, None]
        seen = (at <= p) & ((at > p - case["window"]) | (at < case["sinks"]) if case["window"] else at >= 0)
        lse = st["lse"][start[i]: start[i] + r].double().unflatten(1, (case["heads"], case["group"]))
        old = st["score"][page, :, at % case["page"]].double()
        old[n - r:] = 0.0
        for h in range(case["heads"]):
            w = (x[:, h].reshape(r * case["group"], -1) @ k[:, h].t()).view(r, case["group"], n) / math.sqrt(case["dim"])
            w = torch.exp(w - lse[:, h, :, None]).masked_fill(~seen[:, None], 0.0)
            out[page, h, at % case["page"]] = old[:, h] + w.sum((0, 1))
    return out


def _exact_turned(st, x):
    c = st["case"]
    angle = st["position"].double()[:, None] * st["freq"] * (-1.0 if c["backward"] else 1.0)
    turn = torch.polar(torch.full_like(angle, st["factor"]), angle)[:, None]
    v = x.double()
    part = v[..., : c["part"]]
    part = part.unflatten(-1, (2, -1)).transpose(-1, -2) if c["layout"] == "half" else part.unflatten(-1, (-1, 2))
    z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
    z = z.transpose(-1, -2) if c["layout"] == "half" else z
    return torch.cat([z.reshape(*v.shape[:-1], c["part"]), v[..., c["part"]:]], -1)
