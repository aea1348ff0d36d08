"""The operators on quantized operands from their definitions, in 64 bits on the CPU: byte layouts as
include/gptq.h states them, written element by element, and the bounds their tests hold results
to.  Shares nothing with the library."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}  # below the normal range


# ------------------------------------------------------------------ weights

def weight_values(codes, scale, codec):
    """f64 [rows, n] of a sweep's plane and scales."""
    q = codes.cpu().numpy()
    rows = q.shape[0]
    if codec == "q4tp":
        lev = np.stack([q & 15, q >> 4], -1).reshape(rows, -1).astype(np.float64) - 8.0
    else:
        lev = np.stack([(q >> (2 * i)) & 3 for i in range(4)], -1).reshape(rows, -1).astype(np.float64) - 1.5
    return torch.from_numpy(lev * np.repeat(scale.cpu().numpy().astype(np.float64), 32, axis=1))


def activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def linear(X, codes, scale, codec, bias, act, residual):
    """(y f64, bound): the definition and how far a correct kernel may be from it.

    A group's 32 products of whole numbers up to 32 (code plus operand offset) with x are summed in
    f32 (error at most 2^-23 of the running magnitude an addition; 40 additions, the three-term
    split included), the G scaled sums likewise.  The 16-bit product instead rounds each weight by
    half a step and sums n products.  With either, no activation has a slope over 1.13, and f32
    functions add 2^-20; then one rounding to the type."""
    W = weight_values(codes, scale, codec)
    x = X.double().cpu()
    n = x.shape[1]
    z = x @ W.t()
    S = torch.from_numpy(np.repeat(np.abs(scale.cpu().numpy().astype(np.float64)), 32, axis=1))
    spread, size = x.abs() @ S.t(), x.abs() @ W.abs().t()
    sums = 2.0 ** -23 * (40 * 56 * spread + (n // 32 + 24) * (size + 32 * spread) / 4 + n * size / 4)
    # f32 sums of many terms err as a random walk, not in one direction: 1/4 of the worst case above.
    weight = 0.0 if X.dtype == torch.float32 else HALF[X.dtype]
    err = sums + weight * size
    if bias is not None:
        z = z + bias.double().cpu()
    err = err + 2.0 ** -23 * z.abs()
    y = activate(z, act)
    err = 1.13 * err + 2.0 ** -20 * (y.abs() + z.abs() * (act != "none"))
    if residual is not None:
        y = y + residual.double().cpu()
    return y, err + HALF[X.dtype] * (y.abs() + err) + TINY[X.dtype]


# ------------------------------------------------------------------ the cache

def up5(a):
    """Smallest number of 5 significant bits at or above each a > 0."""
    m, e = np.frexp(a)
    return np.ldexp(np.ceil(m * 32.0), e - 5)


def quantize(x):
    """x [..., D] -> (codes -7..7, scales [..., D / 32]) in f64 / int."""
    v = np.asarray(x, np.float64)
    v = v.reshape(*v.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        a = np.max(np.abs(v), -1)
        bad = ~np.isfinite(v).all(-1) | (a >= 2.0 ** 127)
    a = np.where(bad, 0.0, a)
    s = np.where(a > 0, np.maximum(up5(np.where(a > 0, a, 7.0) / 7.0), 2.0 ** -126), 0.0)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where((s > 0)[..., None], np.rint(v / np.where(s > 0, s, 1.0)[..., None]), 0.0)
    c = np.where(bad[..., None], 0.0, c).astype(np.int64)
    return c.reshape(np.shape(x)), np.where(bad, np.nan, s)


def key_place(d, G):
    """(byte, shift) of a channel in a key's row."""
    i, h, j = d // 32, d % 32 // 8, d % 8
    nibble = j // 2 + 4 * (j % 2)
    return 4 * (h * G + i) + nibble // 2, 4 * (nibble % 2)


def value_place(d, G):
    i, n, m = d // 32, d % 32 // 16, d % 16
    return m * G + i, 4 * n


class Cache:
    """A paged cache in the stated layout, on the CPU: planes as numpy arrays."""

    def __init__(self, pages, page, heads, dim, fill=0):
        self.pages, self.page, self.heads, self.dim, self.G = pages, page, heads, dim, dim // 32
        self.k = np.full((pages, heads, page, dim // 2), fill, np.uint8)
        self.v = self.k.copy()
        self.ks = np.zeros((pages, heads, page, self.G), np.float64)
        self.vs = self.ks.copy()

    def place(self, table, b, pos):
        if pos < 0 or pos >= table.shape[1] * self.page:
            return None
        p = int(table[b, pos // self.page])
        return (p, pos % self.page) if 0 <= p < self.pages else None

    def write(self, table, length, start, K, V):
        for b, r, pos in rows_of(table.shape[0], length, start):
            at = self.place(table, b, pos)
            if at is None:
                continue
            for plane, scales, x, where in ((self.k, self.ks, K, key_place), (self.v, self.vs, V, value_place)):
                c, s = quantize(x[r])
                row = np.zeros((self.heads, self.dim // 2), np.uint8)
                for d in range(self.dim):
                    byte, shift = where(d, self.G)
                    row[:, byte] |= ((c[:, d] + 8) << shift).astype(np.uint8)
                plane[at[0], :, at[1]] = row
                scales[at[0], :, at[1]] = s

    def tensors(self, device):
        t = [torch.from_numpy(self.k.copy()), torch.from_numpy(self.v.copy())]
        s = [torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16) for x in (self.ks, self.vs)]
        return tuple(x.to(device) for x in t + s)

    def values(self, table, b, n):
        """(K, V) f64 [n, heads, dim] of a sequence's first n positions, and which exist."""
        places = [self.place(table, b, pos) for pos in range(min(n, table.shape[1] * self.page))]
        places += [None] * (n - len(places))
        there = np.array([p is not None for p in places], bool).reshape(n)
        p = np.array([x[0] if x else 0 for x in places], np.int64)
        o = np.array([x[1] if x else 0 for x in places], np.int64)
        out = []
        for plane, scales, where in ((self.k, self.ks, key_place), (self.v, self.vs, value_place)):
            m = np.array([where(d, self.G) for d in range(self.dim)])
            c = (plane[p, :, o].astype(np.int64)[..., m[:, 0]] >> m[:, 1]) & 15
            val = (c - 8) * np.repeat(scales[p, :, o], 32, axis=-1)
            out.append(np.where(there[:, None, None], val, 0.0))
        return out[0], out[1], there


def rows_of(seqs, length, start):
    """(sequence, row, position) of every row of a call."""
    for b in range(seqs):
        r0, r1 = (b, b + 1) if start is None else (int(start[b]), int(start[b + 1]))
        for r in range(r0, r1):
            yield b, r, int(length[b]) - (r1 - r0) + (r - r0)


def attention(cache, Q, table, length, start, scale, window, sinks):
    """(O, lse, bound) f64 of the definition.  The bound: a score is a sum of G scaled f32 sums of 32
    products with offset codes (as linear's); an error d of a score moves its weight by e^d - 1; the
    weight is rounded by r (8, 16 or 24 bits, the terms' truncations counted), exp2 and the
    division add 2^-20; sums over the sequence run in f32 as a random walk of their steps at offset
    magnitude; then the rounding to the type."""
    q = Q.double().cpu().numpy()
    group = q.shape[1] // cache.heads
    O = np.zeros(q.shape)
    bound = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    r = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -15, torch.float32: 2.0 ** -22}[Q.dtype]
    done = np.zeros(q.shape[0], bool)
    kv = {}
    for b, row, pos in rows_of(table.shape[0], length, start):
        done[row] = True
        if b not in kv:
            kv[b] = cache.values(table, b, max(0, int(length[b])))
        K, V, there = kv[b]
        n = np.arange(len(there))
        seen = there & (n <= pos)
        if window:
            seen &= (n > pos - window) | (n < sinks)
        if not seen.any():
            continue
        k, v = K[seen].transpose(1, 0, 2), V[seen].transpose(1, 0, 2)          # [heads, n, dim]
        x = q[row].reshape(cache.heads, group, -1)
        s = scale * (x @ k.transpose(0, 2, 1))                                  # [heads, group, n]
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        l = p.sum(-1, keepdims=True)
        w = p / l
        o = w @ v
        d = abs(scale) * 2.0 ** -23 * 40 * 56 * np.abs(k).max(-1)[:, None] * np.abs(x).sum(-1, keepdims=True) / 7
        d = d + 2.0 ** -21 * (np.abs(s) + 2)
        rel = w * (r + 2 * d + 2.0 ** -19)
        acc = 8 * math.sqrt(s.shape[-1] / 32 + 64) * 2.0 ** -24 * 48
        peak = np.repeat(np.abs(v).reshape(*v.shape[:2], -1, 32).max(-1), 32, -1)
        err = rel @ np.abs(v) + rel.sum(-1, keepdims=True) * np.abs(o) + acc * (w @ peak) / 7
        O[row], bound[row] = o.reshape(O[row].shape), err.reshape(O[row].shape)
        lse[row] = (top + np.log(l)).reshape(-1)
    bound += HALF[Q.dtype] * (np.abs(O) + bound) + TINY[Q.dtype]
    return O, lse, bound, done


def assert_within(got, want, bound, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got)
    want, bound = np.asarray(want), np.asarray(bound)
    assert got.shape == want.shape, f"{what}: shape {got.shape}, not {want.shape}"
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    d = np.abs(got - want)[~nan]
    if d.size:
        worst = np.argmax(d - bound[~nan])
        assert (d <= bound[~nan]).all(), f"{what}: off by {d[worst]:.3e}, bound {bound[~nan][worst]:.3e}"
