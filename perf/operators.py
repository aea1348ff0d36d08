"""What is measured of the operators on quantized operands: the product with the sweep's codes
(gptq_linear), the 4-bit cache written and read back (gptq_cache_write, gptq_cache_read), and the
attention over it (gptq_cache_attention).

``run`` computes a case in plain torch operations (``own`` false) or with the framework's calls
(``own`` true), from the same state.  ``exact`` is the definition in 64 bits.

Codes of a weight matrix are the sweeps' planes: q4tp keeps column 2m in the low nibble of byte m
and 2m + 1 in the high one, value (q - 8) s; q2tp keeps column 4m + i in bits 2i of byte m, value
(q - 1.5) s; s is f32, one per row and 32 columns.

The cache keeps c + 8 (c in -7..7) in a nibble, value c s, s one bf16 per token, head and 32
channels.  With G = D / 32 groups, a key's row of D / 2 bytes holds word (h, g) of 4 bytes at
4 (h G + g), h < 4: nibble k of it is channel 32 g + 8 h + 2 k, nibble k + 4 the channel after.  A
value's row holds for each m < 16 the G bytes from m G on: nibble i of byte g is channel
32 g + 16 i + m.  Scales: [pages, heads, page, G].
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
    linear = {"op": "linear", "bias": False, "act": "none", "residual": False}
    cache = {"heads": 8, "dim": 128, "page": 16, "ragged": True}
    return [
        # One token through an attention projection of the 4096-wide layer: latency.
        {"name": "linear_one_token", **linear, "t": 1, "rows": 4096, "n": 4096, "codec": "q4tp", "type": "bf16"},
        # A decode batch through the 17408-wide down projection, added to the residual stream.
        {"name": "linear_decode_13", **linear, "t": 13, "rows": 5120, "n": 17408, "codec": "q4tp", "type": "f16",
         "residual": True},
        # Calibration rows of an odd count through a 2-bit layer in f32, the next layer's inputs.
        {"name": "linear_calibration_f32", **linear, "t": 333, "rows": 2048, "n": 8192, "codec": "q2tp", "type": "f32",
         "bias": True, "act": "gelu"},
        # A whole prompt through the down projection: the largest product.
        {"name": "linear_prompt_4096", **linear, "t": 4096, "rows": 5120, "n": 17408, "codec": "q4tp", "type": "bf16",
         "bias": True, "act": "silu", "residual": True},
        # One new token of each of 48 sequences into the cache, and what it then stands for.
        {"name": "write_decode_48", "op": "write", **cache, "seqs": 48, "rows": 1, "len": 4000, "type": "bf16"},
        # Prompts of up to 4096 tokens into the cache.
        {"name": "write_prompts", "op": "write", **cache, "seqs": 6, "rows": 4096, "len": 4096, "dim": 64, "type": "f16",
         "heads": 10},
        # One short sequence read back for a check.
        {"name": "read_short", "op": "read", **cache, "seqs": 1, "rows": 777, "len": 777, "heads": 4, "type": "f32"},
        # Long sequences read back, to be handed to a dense attention.
        {"name": "read_long", "op": "read", **cache, "seqs": 8, "rows": 8192, "len": 8192, "page": 64, "type": "bf16"},
        # One user, one token, a middling context: latency.
        {"name": "attend_one_1500", "op": "attend", **cache, "seqs": 1, "rows": 1, "len": 1500, "group": 4, "type": "bf16",
         "window": 0, "sinks": 0},
        # A serving batch of single tokens over contexts of up to 4096: the cache's bandwidth.
        {"name": "attend_decode_64", "op": "attend", **cache, "seqs": 64, "rows": 1, "len": 4096, "group": 8,
         "type": "bf16", "window": 0, "sinks": 0},
        # Some drafted tokens a sequence, a sliding window with sinks, 7 query heads to a cached one.
        {"name": "attend_window_drafts", "op": "attend", **cache, "seqs": 16, "rows": 5, "len": 6000, "group": 7, "dim": 64,
         "type": "f16", "window": 1024, "sinks": 4},
        # A chunk of a prompt over what is cached already.
        {"name": "attend_prompt_chunk", "op": "attend", **cache, "seqs": 2, "rows": 2048, "len": 8192, "group": 4, "heads": 4,
         "type": "bf16", "window": 0, "sinks": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "write", "read", "attend", "attend"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "linear":
        t = _log(rng, 1, 4096)
        n = 32 * _log(rng, 8, 544)
        rows = _log(rng, 200, 5120)
        if kind == "f32":
            t = min(t, 1024)
        return {"op": op, "t": t, "rows": rows, "n": n, "codec": rng.choice(["q4tp", "q4tp", "q2tp"]), "type": kind,
                "bias": rng.random() < 0.5, "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                "residual": rng.random() < 0.5}
    case = {"op": op, "heads": rng.randint(1, 12), "dim": rng.choice([64, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
            "ragged": rng.random() < 0.8, "type": kind}
    if op in ("write", "read"):
        rows = _log(rng, 1, 4096)
        seqs = _log(rng, 1, max(1, min(64, 24000 // rows)))
        return {**case, "seqs": seqs, "rows": rows, "len": rows + (_log(rng, 1, 4096) if rng.random() < 0.5 else 0)}
    if rng.random() < 0.6:  # decoding, a few rows a sequence
        rows, group = rng.choice([1, 1, 1, 2, 5]), rng.choice([1, 2, 3, 4, 7, 8, 16])
        seqs = _log(rng, 1, 48)
        length = _log(rng, 16, 4096 if seqs > 12 else 12000)
    else:
        rows, group = _log(rng, 16, 1024), rng.choice([1, 2, 4, 5, 8])
        seqs = rng.randint(1, 3)
        length = rows + _log(rng, 1, 3000)
        case["heads"] = rng.randint(1, 6)
    window = 0 if rng.random() < 0.6 else _log(rng, 8, 2000)
    return {**case, "seqs": seqs, "rows": rows, "len": max(length, rows), "group": group, "window": window,
            "sinks": rng.choice([0, 1, 4, 64]) if window else 0}


# ---------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _lengths(case):
    """Tokens of each sequence and how many of them are rows of this call: sizes, so the case's alone."""
    B, R, L = case["seqs"], case["rows"], case["len"]
    r = np.random.RandomState(31 * B + 17 * R + L)
    if not case["ragged"]:
        return np.full(B, L), np.full(B, R)
    if R == L:  # whole sequences
        n = np.maximum(1, np.round(L * r.uniform(0.4, 1.0, B))).astype(int)
        n[r.randint(B)] = L
        return n, n.copy()
    rows = np.full(B, R) if R <= 8 else np.maximum(1, np.round(R * r.uniform(0.5, 1.0, B))).astype(int)
    n = np.maximum(rows, np.round(L * r.uniform(0.4, 1.0, B)).astype(int))
    n[r.randint(B)] = L
    return n, rows


def _batch(case, seed):
    """Pages of each sequence in an order without pattern, lengths, and the rows' starts."""
    length, rows = _lengths(case)
    r = np.random.RandomState((int(seed) * 131 + 7) % (1 << 31))
    page = case["page"]
    blocks = -(-length // page)
    width, total = int(blocks.max()), int(blocks.sum())
    pages = r.permutation(total + 3)[:total].astype(np.int32)
    table = np.zeros((len(length), width), np.int32)
    table[np.arange(width)[None, :] < blocks[:, None]] = pages
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return {"length": length, "rows": rows, "pages": total + 3, "table": table, "start": start}


def _cache_codes(case, seed, pages):
    """Codes 1..15 and scales of a whole cache, channels in order: what normal keys and values make."""
    g = _gen(seed)
    shape = (pages, case["heads"], case["page"], case["dim"])
    out = []
    for spread in (0.35, 0.15):
        q = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, 2.9, generator=g)
        q = (q.round_().clamp_(-7, 7) + 8).to(torch.uint8)
        z = torch.empty(shape[:3] + (case["dim"] // 32,), dtype=torch.float32, device="cuda").normal_(0.0, 0.3, generator=g)
        s = (z.exp() * spread).view(torch.int32) & ~0x7FFFF  # 5 significant bits
        out += [q, s.view(torch.float32).to(torch.bfloat16)]
    return out


def _pack_keys(q):
    """[..., D] codes in order -> [..., D / 2] bytes of key rows."""
    G = q.shape[-1] // 32
    x = q.view(*q.shape[:-1], G, 4, 4, 2)                       # g, h, k, parity
    x = x.movedim(-4, -3)                                       # h, g, k, parity
    x = torch.cat([x[..., 0], x[..., 1]], -1)                   # h, g, 8 nibbles
    return (x[..., 0::2] | (x[..., 1::2] << 4)).reshape(*q.shape[:-1], G * 16)


def _pack_values(q):
    G = q.shape[-1] // 32
    x = q.view(*q.shape[:-1], G, 2, 16)                         # g, i, m
    return (x[..., 0, :] | (x[..., 1, :] << 4)).transpose(-1, -2).reshape(*q.shape[:-1], G * 16)


def prepare(case, seed):
    kind = TYPES[case["type"]]
    g = _gen(seed + 1)
    if case["op"] == "linear":
        t, rows, n = case["t"], case["rows"], case["n"]
        st = {"case": case}
        # Activations with a few loud channels, as the calibration workloads have.
        loud = torch.where(torch.rand(n, device="cuda", generator=g) < 0.01, 8.0, 1.0)
        st["x"] = (torch.randn(t, n, device="cuda", generator=g) * loud).to(kind)
        if case["codec"] == "q4tp":
            q = (torch.randn(rows, n, device="cuda", generator=g) * 2.9).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
            st["codes"] = q[:, 0::2] | (q[:, 1::2] << 4)
        else:
            q = torch.randint(0, 4, (rows, n), device="cuda", generator=g, dtype=torch.uint8)
            st["codes"] = q[:, 0::4] | (q[:, 1::4] << 2) | (q[:, 2::4] << 4) | (q[:, 3::4] << 6)
        # Rungs of a ladder: 2^(lo + c step), a few octaves in a row.
        lo = -8.5 + torch.rand(rows, 1, device="cuda", generator=g)
        c = torch.randint(0, 32, (rows, n // 32), device="cuda", generator=g)
        st["scale"] = torch.exp2(lo + c * 0.06)
        st["bias"] = torch.randn(rows, device="cuda", generator=g) if case["bias"] else None
        st["residual"] = torch.randn(t, rows, device="cuda", generator=g).to(kind) if case["residual"] else None
        return st
    b = _batch(case, seed)
    total = int(b["start"][-1])
    single = bool((b["rows"] == 1).all())
    st = {"case": case, "rows": total, "width": int(b["length"].max()), "most": int(b["rows"].max()),
          "table": torch.from_numpy(b["table"]).cuda(), "length": torch.from_numpy(b["length"].astype(np.int32)).cuda(),
          "start": torch.from_numpy(b["start"]).cuda(), "single": single}
    H, D = case["heads"], case["dim"]
    if case["op"] == "write":
        shape = (b["pages"], H, case["page"])
        st["cache"] = tuple(torch.zeros(*shape, D // 2, dtype=torch.uint8, device="cuda") if i == 0 else
                            torch.zeros(*shape, D // 32, dtype=torch.bfloat16, device="cuda")
                            for i in (0, 0, 1, 1))
        st["k"], st["v"] = _new_rows(case, seed, total)
        return st
    kq, ks, vq, vs = _cache_codes(case, seed, b["pages"])
    st["cache"] = (_pack_keys(kq), _pack_values(vq), ks, vs)
    if case["op"] == "attend":
        st["q"] = _queries(case, seed, total)
    return st


def _new_rows(case, seed, total):
    """Keys with some loud channels, values without, both slices of one projection's output."""
    g = _gen(seed + 2)
    H, D = case["heads"], case["dim"]
    x = torch.randn(total, 2, H, D, device="cuda", generator=g)
    x[:, 0] *= torch.exp(torch.randn(H, D, device="cuda", generator=g))
    x = x.to(TYPES[case["type"]])
    return x[:, 0], x[:, 1]


def _queries(case, seed, total):
    g = _gen(seed + 3)
    x = torch.randn(total, case["heads"] * case["group"], case["dim"], device="cuda", generator=g)
    return x.to(TYPES[case["type"]])


# ---------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "write": _own_write, "read": _own_read, "attend": _own_attend}[op](state)
    return {"linear": _plain_linear, "write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](state)


def _own_linear(s):
    c = s["case"]
    return _import().gptq_linear(s["x"], s["codes"], s["scale"], codec=c["codec"], bias=s["bias"], act=c["act"],
                                 residual=s["residual"])


def _own_write(s):
    pwq = _import()
    start = None if s["single"] else s["start"]
    pwq.gptq_cache_write(s["cache"], s["k"], s["v"], s["table"], s["length"], start=start)
    return pwq.gptq_cache_read(s["cache"], s["table"], s["length"], start=start, rows=s["rows"],
                               dtype=TYPES[s["case"]["type"]])


def _own_read(s):
    return _import().gptq_cache_read(s["cache"], s["table"], s["length"], start=None if s["single"] else s["start"],
                                     rows=s["rows"], dtype=TYPES[s["case"]["type"]])


def _own_attend(s):
    c = s["case"]
    return _import().gptq_cache_attention(s["cache"], s["q"], s["table"], s["length"],
                                          start=None if s["single"] else s["start"], window=c["window"],
                                          sinks=c["sinks"])


def _plain_linear(s):
    c = s["case"]
    q = s["codes"]
    if c["codec"] == "q4tp":
        w = torch.stack([q & 15, q >> 4], -1).float() - 8.0
    else:
        w = torch.stack([q & 3, (q >> 2) & 3, (q >> 4) & 3, q >> 6], -1).float() - 1.5
    w = w.view(c["rows"], c["n"] // 32, 32) * s["scale"][..., None]
    y = s["x"].float() @ w.view(c["rows"], c["n"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "relu":
        y = torch.clamp_min(y, 0.0)
    elif c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _plain_quantized(x):
    """The values that a row's codes stand for; in 64 bits, for values next to a border."""
    v = x.double().unflatten(-1, (-1, 32))
    a = v.abs().amax(-1, keepdim=True) / 7.0
    bits = (a.view(torch.int64) + ((1 << 48) - 1)) & ~((1 << 48) - 1)
    s = torch.where(a > 0, torch.clamp_min(bits.view(torch.float64), 2.0 ** -126), 0.0)
    c = torch.round(v / torch.where(s > 0, s, 1.0))
    return (c * s).flatten(-2).to(x.dtype)


def _plain_write(s):
    return _plain_quantized(s["k"]), _plain_quantized(s["v"])


def _plain_rows(s):
    """Sequence and position of each row of the call."""
    i = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["start"][1:], i, right=True)
    at = s["length"][b] - (s["start"][b + 1] - s["start"][b]) + (i - s["start"][b])
    return b, at


def _plain_gather(s, b, at):
    """Keys and values, f32, of positions `at` of sequences `b`: two index tensors of one shape."""
    k, v, ks, vs = s["cache"]
    page = k.shape[2]
    p, o = s["table"][b, at // page].long(), (at % page).long()
    G = k.shape[3] // 16
    w = k[p, :, o].unflatten(-1, (4, G, 4))
    w = torch.stack([w & 15, w >> 4], -1).flatten(-2)                  # h, g, nibble
    w = torch.stack([w[..., :4], w[..., 4:]], -1).flatten(-2)          # h, g, channel
    keys = w.transpose(-2, -3).flatten(-2).float() - 8.0               # g, channel of the group
    u = v[p, :, o].unflatten(-1, (16, G)).transpose(-1, -2)            # g, m
    values = torch.stack([u & 15, u >> 4], -2).flatten(-2).float() - 8.0
    keys = keys * ks[p, :, o].float()[..., None]
    values = values * vs[p, :, o].float()[..., None]
    return keys.flatten(-2), values.flatten(-2)


def _plain_read(s):
    k, v = _plain_gather(s, *_plain_rows(s))
    kind = TYPES[s["case"]["type"]]
    return k.to(kind), v.to(kind)


def _plain_attend(s):
    c = s["case"]
    B, H, D, R, L, group = c["seqs"], c["heads"], c["dim"], s["most"], s["width"], c["group"]
    rows = s["start"][1:] - s["start"][:-1]
    pos = torch.arange(L, device="cuda")
    at = torch.minimum(pos[None, :], s["length"][:, None] - 1).long()
    k, v = _plain_gather(s, torch.arange(B, device="cuda")[:, None].expand(B, L), at)   # [B, L, H, D]
    i = torch.arange(R, device="cuda")
    take = torch.minimum(s["start"][:-1, None] + i[None, :], s["start"][1:, None] - 1).long()
    q = s["q"].float()[take].view(B, R, H, group, D).permute(0, 2, 3, 1, 4).reshape(B * H, group * R, D)
    k = k.permute(0, 2, 3, 1).reshape(B * H, D, L)
    v = v.permute(0, 2, 1, 3).reshape(B * H, L, D)
    w = torch.bmm(q, k).mul_(1.0 / math.sqrt(D)).view(B, H, group, R, L)
    p = s["length"][:, None] - rows[:, None] + i[None, :]                                # [B, R]
    seen = pos <= p[..., None]
    if c["window"]:
        seen &= (pos > p[..., None] - c["window"]) | (pos < c["sinks"])
    w.masked_fill_(~seen[:, None, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = torch.bmm(w.view(B * H, group * R, L), v).view(B, H, group, R, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, R, H * group, D)
    return o[i[None, :] < rows[:, None]].to(s["q"].dtype)


# ---------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 4 if case["type"] == "f32" else 2
    if case["op"] == "linear":
        t, rows, n = case["t"], case["rows"], case["n"]
        codes = rows * n // (2 if case["codec"] == "q4tp" else 4)
        out = t * rows * e * (2 if case["residual"] else 1)
        return {"bytes": codes + rows * (n // 32) * 4 + t * n * e + out + (4 * rows if case["bias"] else 0),
                "flops": 2 * t * rows * n}
    length, rows = _lengths(case)
    H, D = case["heads"], case["dim"]
    held = H * D * 2 * (16 + 2) / 32            # a cached token's codes and scales
    dense = H * D * 2 * e                       # its key and value in the call's type
    total = int(rows.sum())
    if case["op"] == "write":
        return {"bytes": int(total * (2 * dense + 2 * held)), "flops": total * H * D * 2 * 4}
    if case["op"] == "read":
        return {"bytes": int(total * (dense + held)), "flops": total * H * D * 2}
    cached, pairs = 0, 0
    for n, r in zip(length.tolist(), rows.tolist()):
        p = np.arange(n - r, n)
        low = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros(r, int)
        pairs += int((p - low + 1 + np.minimum(low, case["sinks"])).sum())
        cached += int(n - low[0] + min(low[0], case["sinks"]))
    return {"bytes": int(cached * held + total * H * case["group"] * D * e * 2),
            "flops": 4 * pairs * H * case["group"] * D}


# ---------------------------------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    if case["op"] == "linear":
        st = prepare(case, seed)
        x, q = st["x"].double(), st["codes"]
        per = 2 if case["codec"] == "q4tp" else 4
        shift = torch.arange(per, device="cuda", dtype=torch.uint8) * (8 // per)
        levels = ((q[:, :, None] >> shift) & (2 ** (8 // per) - 1)).reshape(case["rows"], -1).double()
        levels -= 8.0 if per == 2 else 1.5
        y = x @ (levels * st["scale"].double().repeat_interleave(32, 1)).t()
        y = y + (0.0 if st["bias"] is None else st["bias"].double())
        if case["act"] == "relu":
            y = torch.where(y > 0, y, 0.0)
        if case["act"] == "silu":
            y = y * torch.sigmoid(y)
        if case["act"] == "gelu":
            y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
        if case["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
        return y + (0.0 if st["residual"] is None else st["residual"].double())
    b = _batch(case, seed)
    total = int(b["start"][-1])
    if case["op"] == "write":
        return [_exact_values(x) for x in _new_rows(case, seed, total)]
    kq, ks, vq, vs = _cache_codes(case, seed, b["pages"])
    page = case["page"]

    def sequence(i, q, s):
        """Values [L, H, D] of sequence i, from the cache's codes before they were laid out."""
        pages = torch.from_numpy(b["table"][i, : -(-b["length"][i] // page)].astype(np.int64)).cuda()
        c = (q[pages].double() - 8.0) * s[pages].double().repeat_interleave(32, -1)
        return c.transpose(1, 2).reshape(-1, case["heads"], case["dim"])[: b["length"][i]]

    if case["op"] == "read":
        pairs = [(sequence(i, kq, ks)[-r:], sequence(i, vq, vs)[-r:]) for i, r in enumerate(b["rows"].tolist())]
        return [torch.cat([p[j] for p in pairs]) for j in (0, 1)]
    query, outs = _queries(case, seed, total).double(), []
    for i, (n, r) in enumerate(zip(b["length"].tolist(), b["rows"].tolist())):
        k, v = sequence(i, kq, ks), sequence(i, vq, vs)
        x = query[b["start"][i]: b["start"][i + 1]].unflatten(1, (case["heads"], case["group"]))
        p = torch.arange(n - r, n, device="cuda")[:, None]
        at = torch.arange(n, device="cuda")[None, :]
        seen = (at <= p) & ((at > p - case["window"]) | (at < case["sinks"]) if case["window"] else at >= 0)
        o = torch.empty_like(x)
        for h in range(case["heads"]):
            w = x[:, h].reshape(r * case["group"], -1) @ k[:, h].t() / math.sqrt(case["dim"])
            w = w.view(r, case["group"], n).masked_fill(~seen[:, None], -math.inf)
            o[:, h] = (torch.softmax(w, -1).view(r * case["group"], n) @ v[:, h]).view(r, case["group"], -1)
        outs.append(o.flatten(1, 2))
    return torch.cat(outs)


def _exact_values(x):
    v = x.double().reshape(x.shape[0], x.shape[1], -1, 32)
    a = v.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(a / 7.0)                       # a / 7 = m 2^e, m in [1/2, 1): 5 bits of m, up
    power = ((e.to(torch.int64) + (1023 - 5)) << 52).view(torch.float64)
    s = (torch.ceil(m * 32.0) * power).clamp(min=2.0 ** -126)
    return torch.where(a > 0, torch.round(v / s) * s, 0.0).reshape(x.shape)
