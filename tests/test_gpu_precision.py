"""The operators' sums held to the error model of precision.py, which notices one bf16 term fewer: the
product on codes as whole numbers, at sizes of each of its kernels, and the attention in its two."""
import math

import numpy as np
import pytest
import torch

import precision
from test_gpu_attention import filled
from test_gpu_cache import cuda, sequences
from test_gpu_linear import make

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", [(1, 64, 4096), (3, 64, 4096), (13, 333, 8192), (9, 8200, 4128), (17, 31, 1024), (40, 520, 2176), (64, 48, 4128),
                                      (65, 200, 256), (128, 257, 64), (200, 130, 992), (97, 1411, 2080), (24, 4200, 4224),
                                      (130, 2100, 4128), (333, 515, 8192)])
def test_product(gpu, kind, codec, t, rows, n):
    X, codes, scale, _, _ = make(t, rows, n, kind, codec, t + rows)
    z, sigma = precision.linear(X, codes, scale, codec)
    ok, found = precision.holds(gpu.gptq_linear(X, codes, scale, codec), z, sigma, kind)
    assert ok, found


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lengths,rows,page,heads,group", [([300], [1], 16, 2, 4), ([3000], [1], 16, 1, 8), ([700], [60], 64, 1, 4), ([900, 257], [5, 20], 48, 1, 8),
                                                           ([2200], [150], 32, 1, 4), ([1000, 300, 40], [200, 1, 40], 16, 2, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 40)])
def test_attention(gpu, kind, dim, lengths, rows, page, heads, group, window, sinks):
    table, length, start = sequences(lengths, rows, page, sum(-(-n // page) for n in lengths) + 2, dim)
    cache = filled(int(table.max()) + 3, page, heads, dim, dim)
    Q = torch.randn(int(start[-1]), heads * group, dim, generator=torch.Generator().manual_seed(7)).to(kind).cuda()
    O, lse, sigma = precision.attention(cache, Q, table, length, start, 1.0 / math.sqrt(dim), window, sinks)
    got, l = gpu.gptq_cache_attention(cache.tensors("cuda"), Q, cuda(table), cuda(length), cuda(start), window=window, sinks=sinks,
                                      want_lse=True)
    ok, found = precision.holds(got, O, sigma, kind)
    assert ok, found
    # log of a sum of at least one weight: its terms' errors, the logarithm's, and the sum's rounding.
    assert np.abs(l.cpu().numpy() - lse).max() <= 2.0 ** -19 * (8 + np.abs(lse).max())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("rows,n", [(8205, 608), (1030, 2400)])
def test_exact_weights_at_any_number_of_tokens(gpu, kind, codec, rows, n):
    """The same tokens alone and among 2100, where the weights are rounded unless the caller says otherwise."""
    X, codes, scale, _, _ = make(2100, rows, n, kind, codec, n)
    pick = torch.cat([torch.arange(50), torch.arange(rows - 70, rows)]).cuda()
    z, sigma = precision.linear(X, codes[pick], scale[pick], codec)
    assert gpu.linear_workspace_size(2100, rows, n, kind) > 2 * rows * n     # decoded weights
    ok, found = precision.holds(gpu.gptq_linear(X, codes, scale, codec)[:, pick], z, sigma, kind)
    assert not ok, found
    y = gpu.gptq_linear(X, codes, scale, codec, exact=True)
    ok, found = precision.holds(y[:, pick], z, sigma, kind)
    assert ok, found
    for t in (1, 40, 300):
        few = gpu.gptq_linear(X[:t], codes, scale, codec, exact=True)
        ok, found = precision.holds(few[:, pick], z[:t], sigma[:t], kind)
        assert ok, found
        assert (few == y[:t]).float().mean() > 0.99  # up to the order of f32 sums next to a rounding's border
