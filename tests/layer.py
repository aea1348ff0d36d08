"""The gated block, the gradients, rotary positions and the cache's scores and eviction from their definitions, in 64
bits on the CPU, and the bounds that their tests hold results to.  Shares nothing with the library."""
import math

import numpy as np
import torch

import operands as ref
from operands import HALF, TINY

# Scaled gradients enter the codes' product in 16 bits, f32 in 24: the last term rounded, those before it cut.
TERMS = {torch.bfloat16: 2.0 ** -15, torch.float16: 2.0 ** -15, torch.float32: 2.0 ** -22}
DECODED = 2.0 ** -11  # half a step of a weight decoded to f16


def spans(scale):
    """|s| by column, and each row's largest."""
    s = np.abs(scale.cpu().numpy().astype(np.float64))
    return torch.from_numpy(np.repeat(s, 32, axis=1)), torch.from_numpy(s.max(1))


def sums_bound(spread, size, k):
    """f32 sums of k products, codes with their offset among them, as operands.linear counts them."""
    return 2.0 ** -23 * (40 * 56 * spread + (k // 32 + 24) * (size + 32 * spread) / 4 + k * size / 4)


def product(x, err, W, scale, kind, along):
    """(z, bound) of x W^T (`along` 1) or x W (0), x f64 with an error: sums, and what either way of entering the
    weights rounds.  Decoded weights: half a step of f16, 2^-25 of twice the row's largest scale; activations then
    2^-39 of their largest magnitude, times the row's power of two where they are summed over rows."""
    S, top = spans(scale)
    if along:
        W, S = W.t(), S.t()
    size, spread = x.abs() @ W.abs(), x.abs() @ S
    bound = err @ W.abs() + sums_bound(spread, size, W.shape[0])
    if kind != torch.float32:
        lost = 2.0 ** -24 * top
        bound = bound + DECODED * size + (x.abs().sum(1, keepdim=True) * lost[None, :] if along else (x.abs() @ lost)[:, None])
        # twice the largest scale is the least power that a row has taken out, a level at most 8
        big = (x.abs().amax(1, keepdim=True) if along else (x.abs() * 2 * top).amax(1, keepdim=True))
        bound = bound + 2.0 ** -39 * big * (W.abs().sum(0)[None, :] if along else 8.0 * W.shape[0])
    return x @ W, bound


def linear_backward(dY, codes, scale, codec):
    W = ref.weight_values(codes, scale, codec)
    d = dY.double().cpu()
    z, bound = product(d, TERMS[dY.dtype] * d.abs(), W, scale, dY.dtype, 0)
    return z, bound + HALF[dY.dtype] * (z.abs() + bound) + TINY[dY.dtype]


def slope(a, act):
    if act == "relu":
        return (a > 0).double()
    if act == "silu":
        s = torch.sigmoid(a)
        return s * (1 + a * (1 - s))
    if act == "gelu":
        return 0.5 * torch.special.erfc(-a / math.sqrt(2)) + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(k * (a + 0.044715 * a ** 3))
        return s + a * s * (1 - s) * k * (1 + 3 * 0.044715 * a * a)
    return torch.ones_like(a)


def sums(X, gate, up, codec, biases):
    """((a, bound), (b, bound)) and the matrices."""
    x, out, mats = X.double().cpu(), [], []
    for (codes, scale), bias in zip((gate, up), biases):
        W = ref.weight_values(codes, scale, codec)
        z, err = product(x, torch.zeros_like(x), W, scale, X.dtype, 1)
        if bias is not None:
            z = z + bias.double().cpu()
        out.append((z, err + 2.0 ** -22 * z.abs()))
        mats.append(W)
    return out, mats


def gated(X, gate, up, codec, act, biases):
    """(y, bound): no activation has a slope over 1.13; f32 functions and products add 2^-20."""
    ((a, ea), (b, eb)), _ = sums(X, gate, up, codec, biases)
    f = ref.activate(a, act)
    y = f * b
    bound = 1.13 * ea * (b.abs() + eb) + f.abs() * eb + 2.0 ** -20 * (y.abs() + a.abs() * b.abs() * (act != "none"))
    return y, bound + HALF[X.dtype] * (y.abs() + bound) + TINY[X.dtype]


def gated_backward(dY, X, gate, up, codec, act, biases):
    """(dx, bound).  Second derivatives are below 1.1; relu's slope may be either within the sums' bound of 0.  The
    gradients of a and b are rounded as linear_backward's, or to f16 and to 2^-39 of what bounds them."""
    ((a, ea), (b, eb)), (wg, wu) = sums(X, gate, up, codec, biases)
    d, f, k = dY.double().cpu(), ref.activate(a, act), slope(a, act)
    da, db = d * b * k, d * f
    bend = (a.abs() <= ea).double() if act == "relu" else 1.1 * ea
    eda = d.abs() * (1.13 * eb + (b.abs() + eb) * bend) + 2.0 ** -20 * d.abs() * (b.abs() + eb)
    edb = d.abs() * 1.13 * ea + 2.0 ** -20 * d.abs() * a.abs()
    rough = TERMS[dY.dtype] if dY.dtype == torch.float32 else DECODED
    total, bound = 0.0, 0.0
    for g, e, W, scale in ((da, eda, wg, gate[1]), (db, edb, wu, up[1])):
        z, err = product(g, e + rough * (g.abs() + e), W, scale, dY.dtype, 0)
        total, bound = total + z, bound + err
    if dY.dtype != torch.float32:
        tops = [spans(s)[1] for _, s in (gate, up)]
        wide = [spans(s)[0].sum(1) * (8.0 if codec == "q4tp" else 1.5) for _, s in (gate, up)]
        big = max((2 * tops[0] * wide[1]).max(), (2 * tops[1] * wide[0]).max())
        offset = max([float((2 * t * m.double().cpu().abs()).max()) for t, m in zip(tops, biases) if m is not None], default=0.0)
        most = d.abs().amax(1, keepdim=True) * 1.13 * (X.double().cpu().abs().amax(1, keepdim=True) * big + offset)
        bound = bound + 2.0 ** -39 * most * 8.0 * 2 * d.shape[1]
    return total, bound + HALF[dY.dtype] * (total.abs() + bound) + TINY[dY.dtype]


def rotary(x, position, freq, layout, factor, backward):
    """(y, bound): the angle's fraction of a turn is rounded to f32 (2^-24 of at most half a turn: 2^-23 pi), cosine and
    sine by two units, the products and their sum by one each."""
    v = x.double().cpu()
    half = freq.shape[0]
    angle = position.double().cpu()[:, None] * freq.double().cpu()
    c, s = (factor * f(angle)[:, None] for f in (torch.cos, torch.sin))
    s = -s if backward else s
    i0 = torch.arange(half) if layout == "half" else 2 * torch.arange(half)
    i1 = i0 + (half if layout == "half" else 1)
    y = v.clone()
    a, b = v[..., i0], v[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    bound = torch.zeros_like(y)
    e = abs(factor) * (a.abs() + b.abs()) * (2.0 ** -23 * math.pi + 6 * 2.0 ** -24)
    bound[..., i0] = bound[..., i1] = e
    bound = bound + HALF[x.dtype] * (y.abs() + bound) + TINY[x.dtype]
    bound[..., 2 * half:] = 0.0  # copied
    return y, bound


def score(cache, old, Q, lse, table, length, start, scale, window, sinks):
    """(planes, bound, written): every token of the call's sequences.  A score's error d (as operands.attention
    counts it, and lse's and its own rounding of 2^-22 of their size) moves a weight by e^d - 1, exp2 by 2^-20; sums of
    the rows in f32."""
    q = Q.double().cpu().numpy()
    group = q.shape[1] // cache.heads
    out, bound = old.double().cpu().numpy().copy(), np.zeros(old.shape)
    written = np.zeros(old.shape, bool)
    L = lse.double().cpu().numpy()
    for b in range(table.shape[0]):
        r0, r1 = (b, b + 1) if start is None else (int(start[b]), int(start[b + 1]))
        n = min(max(0, int(length[b])), table.shape[1] * cache.page)
        K, _, there = cache.values(table, b, n)
        first = int(length[b]) - (r1 - r0)
        paid, err = np.zeros((cache.heads, n)), np.zeros((cache.heads, n))
        tok = np.arange(n)
        for r in range(r0, r1):
            pos = first + r - r0
            seen = there & (tok <= pos)
            if window:
                seen &= (tok > pos - window) | (tok < sinks)
            x = q[r].reshape(cache.heads, group, -1)
            k = K.transpose(1, 0, 2)
            s = scale * (x @ k.transpose(0, 2, 1))                        # [heads, group, n]
            l = L[r].reshape(cache.heads, group, 1)
            with np.errstate(over="ignore", invalid="ignore"):
                w = np.where(seen & (l > -np.inf), np.exp(s - np.where(l > -np.inf, l, 0.0)), 0.0)
            d = abs(scale) * 2.0 ** -23 * 40 * np.abs(x) @ np.abs(k).transpose(0, 2, 1)
            d = d + 2.0 ** -21 * (np.abs(s) + np.abs(np.where(l > -np.inf, l, 0.0)) + 2)
            paid += w.sum(1)
            err += (w * (2 * d + 2.0 ** -20)).sum(1)
        for t in range(n):
            at = cache.place(table, b, t)
            if at is None:
                continue
            was = out[at[0], :, at[1]] if t < first else 0.0
            out[at[0], :, at[1]] = was + paid[:, t]
            bound[at[0], :, at[1]] = err[:, t] + 2.0 ** -23 * (math.sqrt(group * (r1 - r0)) + 2) * (paid[:, t] + np.abs(was))
            written[at[0], :, at[1]] = True
    return out, bound, written


def evict(cache, score, table, length, keep, sinks, recent):
    """(length, index [sequences, heads, keep]) of what is kept: sorted by (score, -position), NaN above all, tokens
    without a place below all."""
    seqs = table.shape[0]
    left = np.zeros(seqs, np.int32)
    index = np.full((seqs, cache.heads, keep), -1, np.int32)
    for b in range(seqs):
        n = min(max(0, int(length[b])), table.shape[1] * cache.page)
        left[b] = min(n, keep)
        places = [cache.place(table, b, t) for t in range(n)]
        for h in range(cache.heads):
            if n <= keep:
                index[b, h, :n] = np.arange(n)
                continue
            fixed = list(range(sinks)) + list(range(n - recent, n))

            def rank(t):
                if places[t] is None:
                    return (-1, 0.0, -t)
                x = float(score[places[t][0], h, places[t][1]])
                return (1, 0.0, -t) if math.isnan(x) else (0, x, -t)

            rest = sorted(range(sinks, n - recent), key=rank, reverse=True)[: keep - sinks - recent]
            index[b, h] = sorted(fixed + rest)
    return left, index
