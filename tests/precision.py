"""How far f32 sums may be from the definition, as an error model that sees one bf16 term fewer: the
bounds of operands.py are worst cases, 2^-12 of the sum of magnitudes, and pass a product whose f32
activations have lost their third term.  Independent of the library.

An f32 rounding at magnitude M is off by at most 2^-24 M, 2^-24 M / sqrt(3) in the mean square, and
roundings are taken as independent.  A matrix instruction over 32 products is taken as 4 roundings of
its accumulator (8 products each).  ``sigma`` is the root mean square that this gives for every output;
where the result is f32 its errors have to stay within 1.5 sigma in the mean square (the magnitudes M
are upper estimates; 1.5 is for what is not independent) and 8 sigma one by one (beyond 10^6 normal
values' largest, 5).  Where it is rounded to 16 bits, half a step and 8 sigma.  A term lost moves f32 results by 5
sigma and more (test_precision_host.py does that to both operators)."""
import math

import numpy as np
import torch

from operands import HALF, TINY, rows_of, weight_values

U = 2.0 ** -24 / math.sqrt(3.0)
MFMA = 4                                  # roundings of an accumulator a matrix instruction
TERMS = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}


def linear(X, codes, scale, codec):
    """(z, sigma) f64 of X W^T from codes taken as whole numbers: a group's sum starts at -shift sum x (shift
    = 24 or 5.5) and ends at sum (q - z) x; its accumulator stays below shift (|sum x| + |x|).  Roundings of
    a group: of the start (terms of it, or as many additions) and of the product, one instruction a term
    each.  The G scaled sums are added at the magnitude of their running sum."""
    W = weight_values(codes, scale, codec)
    x = X.double().cpu()
    t, n = x.shape
    shift, level = (24.0, 4.6) if codec == "q4tp" else (5.5, 1.12)   # level: root mean square of q - z
    g = x.view(t, n // 32, 32)
    norm, total = g.norm(dim=-1), g.sum(-1).abs()
    s = scale.double().cpu().abs()
    per = math.sqrt(2 * TERMS[X.dtype] * MFMA) * U * shift
    var = ((per * (total + norm)) ** 2) @ (s ** 2).t()
    run = (norm ** 2) @ (level * s).t() ** 2
    return x @ W.t(), torch.sqrt(var + (n // 32 + 16) * U ** 2 * run)


def linear_rounded(X, codes, scale, codec):
    """(z, sigma) f64 on weights rounded to X's 16-bit type: half a step a weight at most, and one sum of n
    products in the accumulator, MFMA roundings for every 32."""
    W = weight_values(codes, scale, codec)
    x = X.double().cpu()
    size = (x ** 2) @ (W ** 2).t()
    return x @ W.t(), torch.sqrt(size * ((HALF[X.dtype] / math.sqrt(3.0)) ** 2 + (MFMA * x.shape[1] / 32 + 16) * U ** 2))


def attention(cache, Q, table, length, start, scale, window=0, sinks=0):
    """(O, lse, sigma) f64.  A score is G scaled sums of 32 products of codes with q (as linear's, without an
    offset in f32), or one sum of all in the tile kernel; the weight of a token errs by the score's
    error, the exponent's rounding (scores within 8 powers of two above the running maximum, and the factor
    scale log2 e), exp2 (two steps) and its rounding to 8, 16 or 24 bits.  An output errs by its weights'
    errors, independent from token to token, and by the roundings of n / 32 steps at its running magnitude,
    offset included."""
    q = Q.double().cpu().numpy()
    heads, G, terms = cache.heads, cache.G, TERMS[Q.dtype]
    group = q.shape[1] // heads
    shift = 24.0 if terms < 3 else 8.0
    bits = {1: 2.0 ** -8, 2: 2.0 ** -16, 3: 2.0 ** -24}[terms] / math.sqrt(3.0)
    O, sigma, lse = np.zeros(q.shape), np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    kept = {}
    for b, row, pos in rows_of(table.shape[0], length, start):
        if b not in kept:
            kept[b] = cache.values(table, b, int(length[b]))
        K, V, there = kept[b]
        n = np.arange(len(there))
        seen = there & (n <= pos)
        if window:
            seen &= (n > pos - window) | (n < sinks)
        k, v = K[seen].transpose(1, 0, 2), V[seen].transpose(1, 0, 2)            # [heads, n, dim]
        x = q[row].reshape(heads, group, -1)
        s = scale * (x @ k.transpose(0, 2, 1))                                    # [heads, group, n]
        top = s.max(-1, keepdims=True)
        w = np.exp(s - top)
        l = w.sum(-1, keepdims=True)
        w = w / l
        o = w @ v
        xg = x.reshape(heads, group, G, 32)
        size = np.abs(xg.sum(-1)) + np.sqrt((xg ** 2).sum(-1))                     # [heads, group, G]
        ks = np.abs(k).reshape(heads, -1, G, 32).max(-1) / 7.0                     # [heads, n, G], at most a scale
        each = np.sqrt(2 * terms * MFMA) * U * shift
        var = abs(scale) ** 2 * np.einsum("hgi,hni->hgn", (each * size) ** 2, ks ** 2)
        run = abs(scale) ** 2 * np.einsum("hgi,hni->hgn", (4.6 * size) ** 2, ks ** 2)
        var = var + (terms * MFMA * G) * U ** 2 * run
        rel = var + (U * (top - s + 8.0)) ** 2 + (U * s) ** 2 + (4 * U) ** 2 + bits ** 2
        vs = np.abs(v).reshape(heads, -1, G, 32).max(-1).repeat(32, -1) / 7.0       # [heads, n, dim]
        steps = terms * MFMA * (v.shape[1] / 32 + 8)
        spread = np.sqrt((w ** 2) @ (v ** 2))
        offset = (shift * (w @ vs)) ** 2 if terms < 3 else 0.0
        dv = (w ** 2 * rel) @ (v ** 2) + ((w ** 2 * rel).sum(-1, keepdims=True)) * o ** 2
        err = dv + steps * U ** 2 * ((np.abs(o) + spread) ** 2 + offset) + (3 * U * o) ** 2
        O[row], sigma[row] = o.reshape(O[row].shape), np.sqrt(err).reshape(O[row].shape)
        lse[row] = (top + np.log(l)).reshape(-1)
    return O, lse, sigma


def holds(got, want, sigma, kind):
    """Whether results of `kind` are as near as the model says: (they are, what was found)."""
    got, want, sigma = (np.asarray(x.double().cpu() if isinstance(x, torch.Tensor) else x) for x in (got, want, sigma))
    d, sigma = np.abs(got - want), sigma + TINY[kind] * 2.0 ** -20
    if kind is torch.float32:
        ratio = d / (sigma + 2.0 ** -24 * np.abs(want) + TINY[kind])
        rms, most = float(np.sqrt((ratio ** 2).mean())), float(ratio.max())
        return rms <= 1.5 and most <= 8.0, f"{rms:.2f} sigma in the mean square, {most:.2f} at most"
    over = d - HALF[kind] * (np.abs(want) + 8 * sigma) - 8 * sigma - TINY[kind]
    return bool((over <= 0).all()), f"{float((d / (HALF[kind] * np.abs(want) + 8 * sigma + TINY[kind])).max()):.2f} of the bound"
