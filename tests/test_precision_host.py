"""The error model of precision.py: it takes f32 sums done right, and rejects results that lack one bf16
term of the activations, of the queries or of the softmax weights, or whose weights were rounded."""
import math

import numpy as np
import pytest
import torch

import operands as ref
import precision
from test_gpu_attention import filled
from test_gpu_cache import sequences

SIZES = [(3, 64, 4096), (17, 31, 1024), (64, 48, 4128), (65, 200, 256), (128, 257, 64), (200, 130, 992)]


def terms(x, n):
    """x cut to n terms of 8 bits, as truncation leaves them."""
    x = np.asarray(x, np.float32)
    out = np.zeros_like(x)
    for _ in range(n):
        out += ((x - out).view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
    return out.astype(np.float64)


def product(t, rows, n, kind, codec, seed):
    g = torch.Generator().manual_seed(seed)
    X = (torch.randn(t, n, generator=g) * torch.where(torch.rand(n, generator=g) < 0.03, 20.0, 1.0)).to(kind)
    codes = torch.randint(0, 256, (rows, n // (2 if codec == "q4tp" else 4)), generator=g, dtype=torch.uint8)
    return X, codes, torch.exp2(torch.randn(rows, n // 32, generator=g) * 0.5 - 6.0)


@pytest.mark.parametrize("kind", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", SIZES)
def test_linear_model(kind, codec, t, rows, n):
    X, codes, scale = product(t, rows, n, kind, codec, t)
    z, sigma = precision.linear(X, codes, scale, codec)
    W = ref.weight_values(codes, scale, codec)
    right = sum((X.float()[:, i:i + 32] @ W.float()[:, i:i + 32].t()) for i in range(0, n, 32))
    ok, found = precision.holds(right.to(kind), z, sigma, kind)
    assert ok, found
    if kind is not torch.bfloat16:  # one term fewer
        less = torch.from_numpy(terms(X.float().numpy(), precision.TERMS[kind] - 1)) @ W.t()
        ok, found = precision.holds(less.float().to(kind), z, sigma, kind)
        assert not ok, found
    else:                           # weights rounded to the type
        ok, found = precision.holds((X.double() @ W.to(kind).double().t()).float().to(kind), z, sigma, kind)
        assert not ok or t * rows < 1000, found


ATTENTION = [([300], [1], 16, 2, 4), ([700], [60], 64, 1, 4), ([40, 257], [5, 20], 48, 1, 8)]


@pytest.mark.parametrize("kind", [torch.float32, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention_model(kind, dim, case):
    lengths, rows, page, heads, group = ATTENTION[case]
    table, length, start = sequences(lengths, rows, page, sum(-(-n // page) for n in lengths) + 2, case)
    cache = filled(int(table.max()) + 3, page, heads, dim, case)
    Q = torch.randn(int(start[-1]), heads * group, dim, generator=torch.Generator().manual_seed(case)).to(kind)
    O, _, sigma = precision.attention(cache, Q, table, length, start, 1.0 / math.sqrt(dim))
    full = precision.TERMS[kind]

    def run(qterms, pterms):
        out = np.zeros(O.shape)
        q = terms(Q.float().numpy(), qterms)
        for b, row, pos in ref.rows_of(len(lengths), length, start):
            K, V, _ = cache.values(table, b, int(length[b]))
            k, v = K[:pos + 1].transpose(1, 0, 2), V[:pos + 1].transpose(1, 0, 2)
            s = q[row].reshape(heads, group, dim) @ k.transpose(0, 2, 1) / math.sqrt(dim)
            e = np.exp(s - s.max(-1, keepdims=True))
            # The weights' last term is rounded, the ones before are cut.
            p = terms(e, pterms - 1)
            p = p + torch.from_numpy((e - p).astype(np.float32)).to(torch.bfloat16).double().numpy()
            out[row] = ((p @ v) / e.sum(-1, keepdims=True)).reshape(out[row].shape)
        return torch.from_numpy(out).to(torch.float32).to(kind)

    ok, found = precision.holds(run(full, full), O, sigma, kind)
    assert ok, found
    for less in ((full - 1, full), (full, full - 1)):
        ok, found = precision.holds(run(*less), O, sigma, kind)
        assert not ok, (less, found)
