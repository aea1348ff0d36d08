"""Calls of the operators on quantized operands that their other tests do not make: outputs over inputs, tensors
that require gradients, infinities, activations far from zero, scales far apart, long captured attentions."""
import pytest
import torch

import operands as ref
import precision
from test_gpu_attention import filled
from test_gpu_cache import cuda, sequences
from test_gpu_linear import make

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 40, 300])
def test_out_over_x(gpu, t):
    """A square layer into its own input raises and leaves it alone; into another slice of its buffer it runs."""
    X, codes, scale, _, _ = make(t, 256, 256, torch.bfloat16, "q4tp", t)
    keep = X.clone()
    with pytest.raises(gpu.GptqError):
        gpu.gptq_linear(X, codes, scale, out=X)
    assert torch.equal(X, keep)
    both = torch.zeros(t, 512, dtype=X.dtype, device="cuda")
    both[:, 256:] = X
    gpu.gptq_linear(both[:, 256:], codes, scale, out=both[:, :256])
    assert torch.equal(both[:, :256], gpu.gptq_linear(X, codes, scale)) and torch.equal(both[:, 256:], X)


@pytest.mark.gpu
def test_gradients_are_refused_not_dropped(gpu):
    X, codes, scale, bias, _ = make(3, 40, 64, torch.float32, "q4tp", 1)
    want = gpu.gptq_linear(X, codes, scale, bias=bias)
    for kw in (dict(X=X.clone().requires_grad_()), dict(bias=bias.clone().requires_grad_()), dict(scale=scale.clone().requires_grad_())):
        args = dict(X=X, codes=codes, scale=scale, bias=bias)
        args.update(kw)
        with pytest.raises(ValueError):
            gpu.gptq_linear(**args)
        with torch.no_grad():
            assert torch.equal(gpu.gptq_linear(**args), want)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,rows,n", [(5, 70, 128), (40, 520, 2176), (300, 515, 1504), (1100, 8205, 608)])
def test_a_token_with_an_infinity(gpu, act, kind, t, rows, n):
    """NaN, or the activation of an infinite sum with the weight's sign, and nothing else; a NaN's token is NaN
    throughout; other tokens have the bits they have without either."""
    X, codes, scale, bias, _ = make(t, rows, n, kind, "q4tp", t)
    clean = gpu.gptq_linear(X, codes, scale, "q4tp", bias, act)
    bad = X.clone()
    bad[1, 7], bad[t - 2, n - 1] = float("nan"), float("inf")
    y = gpu.gptq_linear(bad, codes, scale, "q4tp", bias, act)
    others = [i for i in range(t) if i not in (1, t - 2)]
    assert torch.equal(y[others], clean[others])
    assert torch.isnan(y[1]).all()
    level = (codes[:, -1] >> 4).int() - 8           # the weight that meets the infinity
    down = {"none": float("-inf"), "relu": 0.0}.get(act, float("nan"))
    want = torch.where(level > 0, float("inf"), torch.where(level < 0, down, float("nan"))).to(kind)
    got = y[t - 2]
    assert (torch.isnan(got) | (got == want)).all()


@pytest.mark.gpu
def test_scales_far_below_their_rows_largest(gpu):
    """f16, many tokens: a group 2^-30 of its row's largest is lost beside it, and is not with exact weights."""
    t, rows, n = 1100, 8205, 608
    X, codes, scale, _, _ = make(t, rows, n, torch.float16, "q4tp", 3)
    X[:, :32] = 0
    pick = torch.arange(100)
    z, sigma = precision.linear(X, codes[pick], scale[pick], "q4tp")
    scale[:, 0] = 2.0 ** 25
    ok, found = precision.holds(gpu.gptq_linear(X, codes, scale, exact=True)[:, pick.cuda()], z, sigma, torch.float16)
    assert ok, found
    assert gpu.gptq_linear(X, codes, scale).abs().max() < 1e-3 * z.abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,rows,n", [(2, 24000, 64), (40, 24000, 64), (300, 24000, 1024)])
def test_activations_far_from_zero(gpu, act, kind, t, rows, n):
    """The activation of a known z (X = 0, so the bias) to a few f32 steps of its own size, also where it is
    small: |z|^2 (2 |u| for the exponential of 2 u) multiplies the argument's rounding there."""
    z = torch.linspace(-13.0, 13.0, rows)
    y = gpu.gptq_linear(torch.zeros(t, n, dtype=kind, device="cuda"), torch.zeros(rows, n // 2, dtype=torch.uint8, device="cuda"),
                        torch.ones(rows, n // 32, device="cuda"), "q4tp", z.cuda(), act)
    want = ref.activate(z.double(), act)
    steps = 2.0 ** -22 * (4 + z.double() ** 2 * (1 + 0.08 * z.double().abs()))
    # z / (1 + e^w): from w = 128 log 2 on the exponential is infinite in f32 and the quotient 0, off by
    # |z| / (1 + e^w) < |z| 2^-128.
    bound = (steps + ref.HALF[kind]) * want.abs() + ref.TINY[kind] + z.double().abs() * 2.0 ** -128
    ref.assert_within(y, want.expand(t, -1), bound.expand(t, -1), act)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [[1, 1], [300, 40], [1, 600]])
def test_captured_attention_in_pieces(gpu, rows):
    """Long sequences cut into pieces, two calls in a graph: new queries, lengths and pages at every replay."""
    table, length, start = sequences([4000, 2500], rows, 16, 450, 3)
    cache = filled(450, 16, 2, 128, 3)
    planes, tb, st = cache.tensors("cuda"), cuda(table), cuda(start)
    ln = cuda(length)
    total = int(start[-1])
    Q = torch.randn(total, 8, 128, device="cuda").bfloat16()

    def call():
        return (gpu.gptq_cache_attention(planes, Q, tb, ln, st, want_lse=True) +
                gpu.gptq_cache_attention(planes, Q, tb, ln, st, window=1000, sinks=4, want_lse=True))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    g = torch.Generator("cuda").manual_seed(3)
    for i in range(6):
        Q.copy_(torch.randn(Q.shape, device="cuda", generator=g))
        ln.copy_(cuda(length - 400 * i))
        tb.copy_(tb.flip(0) if i % 2 else tb)
        graph.replay()
        got = [o.clone() for o in out]
        want = call()
        if i % 2:
            torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


@pytest.mark.gpu
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", [(5, 70, 128), (300, 515, 1504), (1100, 8205, 608)])
def test_subnormal_activations(gpu, codec, t, rows, n):
    """f16 activations below its normal range count like others (f16 scales large, so that outputs are normal)."""
    X, codes, scale, _, _ = make(t, rows, n, torch.float16, codec, t)
    X = (X.clamp(-8, 8).float() * 2.0 ** -18).half()     # multiples of 2^-24 below 2^-14: all but a few subnormal
    assert (X.abs() < 2.0 ** -14).float().mean() > 0.9 and (X != 0).float().mean() > 0.9
    scale *= 2.0 ** 12
    pick = torch.cat([torch.arange(50), torch.arange(rows - 20, rows)])
    z, sigma = (precision.linear_rounded if t == 1100 else precision.linear)(X, codes[pick], scale[pick], codec)
    ok, found = precision.holds(gpu.gptq_linear(X, codes, scale, codec)[:, pick.cuda()], z, sigma, torch.float16)
    assert ok, found


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
def test_single_rows_beside_a_prompt(gpu, kind):
    """A batch of both kinds: single rows and a long chunk in one call hold the same model as apart."""
    lengths, rows = [300, 40, 700, 1, 900], [1, 1, 400, 1, 3]
    table, length, start = sequences(lengths, rows, 16, 130, 9)
    cache = filled(130, 16, 2, 64, 9)
    Q = torch.randn(int(start[-1]), 8, 64, generator=torch.Generator().manual_seed(9)).to(kind).cuda()
    planes, tb, ln = cache.tensors("cuda"), cuda(table), cuda(length)
    O, _, sigma = precision.attention(cache, Q, table, length, start, 0.125)
    got = gpu.gptq_cache_attention(planes, Q, tb, ln, cuda(start))
    ok, found = precision.holds(got, O, sigma, kind)
    assert ok, found
    for b, r in enumerate(rows):
        own = gpu.gptq_cache_attention(planes, Q[start[b]:start[b + 1]], tb[b:b + 1], ln[b:b + 1], cuda(start[b:b + 2] - start[b]))
        ok, found = precision.holds(own, O[start[b]:start[b + 1]], sigma[start[b]:start[b + 1]], kind)
        assert ok, (b, found)
