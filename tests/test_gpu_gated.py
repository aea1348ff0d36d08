"""The gated block and the gradients of products with codes against their definitions in 64 bits: types, codecs, sizes
from one token and one row up, on codes and on decoded weights, strides, extreme scales, values that are not finite,
differences, other streams and captured graphs."""
import pytest
import torch

import layer
import operands as ref

TYPES = [torch.bfloat16, torch.float16, torch.float32]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# On codes: one launch, pieces, ragged groups, rows and tokens.
SMALL = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (15, 33, 128), (16, 64, 160), (17, 31, 1024), (31, 100, 480), (33, 7, 2080),
         (64, 48, 4128), (65, 200, 256), (127, 129, 544), (128, 257, 64), (200, 130, 992), (300, 515, 1504), (97, 1411, 2080)]
# Enough to multiply for decoded weights in 16 bits.
LARGE = [(300, 2101, 2080), (513, 1032, 2592), (2100, 1030, 608), (260, 8200, 640), (777, 520, 3104)]
DENSE = [(1210, 2101, 2080), (600, 4100, 2144), (3300, 1030, 1568)]


def weights(rows, n, codec, g, spread=0.5):
    codes = torch.randint(0, 256, (rows, n // (2 if codec == "q4tp" else 4)), generator=g, dtype=torch.uint8)
    return codes.cuda(), torch.exp2(torch.randn(rows, n // 32, generator=g) * spread - 6.0).cuda()


def make(t, rows, n, kind, codec, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(t, n, generator=g) * torch.where(torch.rand(n, generator=g) < 0.03, 20.0, 1.0)
    dY = torch.randn(t, rows, generator=g) * torch.exp2(torch.randn(t, 1, generator=g) * 3 - 8)
    bias = [torch.randn(rows, generator=g).cuda() for _ in range(2)]
    return X.to(kind).cuda(), dY.to(kind).cuda(), weights(rows, n, codec, g, spread), weights(rows, n, codec, g, spread), bias


def check_back(gpu, dY, w, codec, what="", **kw):
    x = gpu.gptq_linear_backward(dY, *w, codec, **kw)
    want, bound = layer.linear_backward(dY, *w, codec)
    assert x.dtype == dY.dtype
    ref.assert_within(x, want, bound, what)
    return x


def check_gated(gpu, X, gate, up, codec, act, bias=(None, None), what="", **kw):
    y = gpu.gptq_gated(X, gate, up, codec, act, *bias, **kw)
    want, bound = layer.gated(X, gate, up, codec, act, bias)
    ref.assert_within(y, want, bound, what)
    return y


def check_grad(gpu, dY, X, gate, up, codec, act, bias=(None, None), what="", **kw):
    x = gpu.gptq_gated_backward(dY, X, gate, up, codec, act, *bias, **kw)
    want, bound = layer.gated_backward(dY, X, gate, up, codec, act, bias)
    ref.assert_within(x, want, bound, what)
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", SMALL + LARGE + DENSE)
def test_sizes(gpu, kind, codec, t, rows, n):
    X, dY, gate, up, bias = make(t, rows, n, kind, codec, t * 7 + rows)
    check_back(gpu, dY, gate, codec, "linear")
    check_gated(gpu, X, gate, up, codec, "silu", what="gated")
    check_gated(gpu, X, gate, up, codec, "gelu", bias, "gated, biases")
    check_grad(gpu, dY, X, gate, up, codec, "silu", what="gradient")
    check_grad(gpu, dY, X, gate, up, codec, "gelu_tanh", bias, "gradient, biases")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,rows,n", [(3, 130, 288), (260, 130, 288), (300, 2056, 2112), (1210, 2056, 2112)])
def test_activations(gpu, act, kind, t, rows, n):
    X, dY, gate, up, bias = make(t, rows, n, kind, "q4tp", 5)
    for b in ((None, None), bias, (bias[0], None), (None, bias[1])):
        check_gated(gpu, X, gate, up, "q4tp", act, b, act)
        check_grad(gpu, dY, X, gate, up, "q4tp", act, b, act)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,rows,n", [(1, 75, 224), (5, 75, 224), (300, 76, 224), (300, 2051, 2144), (401, 1601, 2080), (1301, 2051, 2144), (1211, 2080, 2144)])
def test_strides(gpu, kind, t, rows, n):
    """Padded rows of every argument, at addresses that keep vectors aligned and not: own columns alone are read and
    written."""
    X, dY, gate, up, bias = make(t, rows, n, kind, "q4tp", 9)
    nan = float("nan")
    for pad, at in ((64, 32), (9, 4), (7, 3)):
        wide = torch.full((t, n + 64), nan, dtype=kind, device="cuda")
        wide[:, 32:32 + n] = X
        d = torch.full((t, rows + pad), nan, dtype=kind, device="cuda")
        d[:, at:at + rows] = dY
        y, x = (torch.full((t, w + pad), 3.0, dtype=kind, device="cuda") for w in (rows, n))
        check_gated(gpu, wide[:, 32:32 + n], gate, up, "q4tp", "silu", bias, out=y[:, at:at + rows])
        check_grad(gpu, d[:, at:at + rows], wide[:, 32:32 + n], gate, up, "q4tp", "silu", bias, out=x[:, at:at + n])
        for z, w in ((y, rows), (x, n)):
            assert (z[:, :at] == 3).all() and (z[:, at + w:] == 3).all()
        x.fill_(3.0)
        check_back(gpu, d[:, at:at + rows], gate, "q4tp", out=x[:, at:at + n])
        assert (x[:, :at] == 3).all() and (x[:, at + n:] == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,rows,n", [(4, 64, 256), (300, 2112, 2112), (1210, 2112, 2112)])
def test_scales_of_any_size(gpu, kind, t, rows, n):
    """Rows whose scales lie many octaves apart, or are zero: every row's share at its own precision in the forward
    products, the large ones' in the gradients."""
    X, dY, gate, up, _ = make(t, rows, n, kind, "q4tp", 11, spread=2.0)
    low, high = (-16, 0) if kind is torch.float16 else (-40, 20)
    for w, flip in ((gate, False), (up, True)):
        ladder = torch.exp2(torch.linspace(low, high, rows, device="cuda").round())[:, None]
        w[1].mul_(ladder.flip(0) if flip else ladder)
        w[1][5] = 0.0
        w[1][6, ::2] = 0.0
    X = (X * 0.125).to(kind)
    for act in ("none", "silu"):
        y, bound = layer.gated(X, gate, up, "q4tp", act, (None, None))
        fine = y.abs() < (30000.0 if kind is torch.float16 else 1e37)
        got = gpu.gptq_gated(X, gate, up, "q4tp", act).cpu()
        ref.assert_within(got[fine], y[fine], bound[fine], act)
    assert fine.float().mean() > 0.9
    check_back(gpu, dY, up, "q4tp")
    check_grad(gpu, dY, X, gate, up, "q4tp", "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("t,rows,n", [(40, 130, 288), (400, 1601, 2080), (1211, 2101, 2080)])
def test_tokens_far_apart(gpu, t, rows, n):
    """bf16 tokens of 2^-60 to 2^60, whose gradients pass f16's range in both directions."""
    X, dY, gate, up, _ = make(t, rows, n, torch.bfloat16, "q4tp", 3)
    X *= torch.exp2(torch.linspace(-30, 20, t, device="cuda").round())[:, None].to(torch.bfloat16)
    dY *= torch.exp2(torch.linspace(60, -60, t, device="cuda").round())[:, None].to(torch.bfloat16)
    check_back(gpu, dY, gate, "q4tp")
    check_gated(gpu, X, gate, up, "q4tp", "relu")
    check_grad(gpu, dY, X, gate, up, "q4tp", "none")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,rows,n", [(20, 130, 288), (300, 2101, 2080), (1210, 2101, 2080)])
def test_values_that_are_not_finite(gpu, kind, t, rows, n):
    """They stay in their tokens."""
    X, dY, gate, up, _ = make(t, rows, n, kind, "q4tp", 21)
    calls = [(dY, lambda: gpu.gptq_linear_backward(dY, *gate)), (X, lambda: gpu.gptq_gated(X, gate, up)),
             (X, lambda: gpu.gptq_gated_backward(dY, X, gate, up)), (dY, lambda: gpu.gptq_gated_backward(dY, X, gate, up))]
    others = [i for i in range(t) if i not in (2, t - 3)]
    for z, call in calls:
        clean, keep = call(), z.clone()
        z[2, 7], z[t - 3, 5] = float("nan"), float("inf")
        bad = call()
        assert torch.equal(bad[others], clean[others])
        assert not torch.isfinite(bad[2]).any() and not torch.isfinite(bad[t - 3]).all()
        z.copy_(keep)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(gpu, act):
    """f32: differences of the forward call along a direction, with what its own bounds and the definition's
    own difference leave open."""
    X, dY, gate, up, bias = make(6, 70, 160, torch.float32, "q4tp", 31)
    g = torch.Generator().manual_seed(1)
    v = torch.randn(6, 160, generator=g).cuda()
    h = 2.0 ** -8
    dx = gpu.gptq_gated_backward(dY, X, gate, up, "q4tp", act, *bias)
    ends = [X + h * v, X - h * v]
    d = dY.double().cpu()
    got, exact, open_ = 0.0, 0.0, 0.0
    for x, sign in zip(ends, (1, -1)):
        y, bound = layer.gated(x, gate, up, "q4tp", act, bias)
        got += sign * (gpu.gptq_gated(x, gate, up, "q4tp", act, *bias).double().cpu() * d).sum() / (2 * h)
        exact += sign * (y * d).sum() / (2 * h)
        open_ += (bound * d.abs()).sum() / (2 * h)
    want, bound = layer.gated_backward(dY, X, gate, up, "q4tp", act, bias)
    w = v.double().cpu()
    along = (dx.double().cpu() * w).sum()
    assert abs(along - got) <= open_ + abs(exact - (want * w).sum()) + (bound * w.abs()).sum()
    assert abs(along) > 20 * abs(along - got)


@pytest.mark.gpu
@pytest.mark.parametrize("t,rows,n", [(37, 2048, 2048), (16, 1024, 2048), (333, 1024, 1024)])
def test_f32_keeps_its_bits(gpu, t, rows, n):
    """Errors over the whole result: a step of 32 rows adds sums whose offset codes are some 12 times the result's
    share of it, rounded by 2^-24 up to 64 times, independently: 12 * 8 / sqrt(3) = 55 units, 2^-18 in all.  A lost third
    term is off by 2^-16 and more."""
    X, dY, gate, up, bias = make(t, rows, n, torch.float32, "q4tp", 41)
    for got, want in ((gpu.gptq_linear_backward(dY, *gate), layer.linear_backward(dY, *gate, "q4tp")[0]),
                      (gpu.gptq_gated(X, gate, up, "q4tp", "silu", *bias), layer.gated(X, gate, up, "q4tp", "silu", bias)[0]),
                      (gpu.gptq_gated_backward(dY, X, gate, up), layer.gated_backward(dY, X, gate, up, "q4tp", "silu", (None, None))[0])):
        e = got.double().cpu() - want
        assert float(e.norm() / want.norm()) < 2.0 ** -18


@pytest.mark.gpu
@pytest.mark.parametrize("t,rows,n", [(400, 1601, 2080), (1210, 2101, 2080)])
def test_decoded_weights_keep_more_bits_than_bf16(gpu, t, rows, n):
    """On weights of 11 bits a bf16 result is off by its own rounding, 2^-9 / sqrt(3) of its binade's top at most: with
    weights of 8 bits it would be 1.4 times that and more."""
    X, dY, gate, up, _ = make(t, rows, n, torch.bfloat16, "q4tp", 51)
    for got, want in ((gpu.gptq_linear_backward(dY, *gate), layer.linear_backward(dY, *gate, "q4tp")[0]),
                      (gpu.gptq_gated(X, gate, up), layer.gated(X, gate, up, "q4tp", "silu", (None, None))[0]),
                      (gpu.gptq_gated_backward(dY, X, gate, up), layer.gated_backward(dY, X, gate, up, "q4tp", "silu", (None, None))[0])):
        own = (want.to(torch.bfloat16).double() - want).norm()
        assert float((got.double().cpu() - want).norm()) < 1.2 * float(own)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
def test_exact_weights(gpu, kind, codec):
    """A size that would decode them for the gradients: results off by less than decoded weights would make them (f16), and the
    definition's bounds for all."""
    t, rows, n = 1210, 2101, 2080
    X, dY, gate, up, bias = make(t, rows, n, kind, codec, 55)
    for got, want in ((check_back(gpu, dY, gate, codec, exact=True), layer.linear_backward(dY, *gate, codec)[0]),
                      (check_gated(gpu, X, gate, up, codec, "silu", bias, exact=True), layer.gated(X, gate, up, codec, "silu", bias)[0]),
                      (check_grad(gpu, dY, X, gate, up, codec, "silu", bias, exact=True),
                       layer.gated_backward(dY, X, gate, up, codec, "silu", bias)[0])):
        own = (want.to(kind).double() - want).norm()
        if kind is not torch.float32:
            assert float((got.double().cpu() - want).norm()) < 1.1 * float(own)


@pytest.mark.gpu
def test_the_same_matrix_twice_and_no_tokens(gpu):
    X, dY, gate, _, bias = make(9, 40, 96, torch.bfloat16, "q4tp", 61)
    check_gated(gpu, X, gate, gate, "q4tp", "none", (bias[0], bias[0]))
    check_grad(gpu, dY, X, gate, gate, "q4tp", "none", (bias[0], bias[0]))
    assert gpu.gptq_gated(X[:0], gate, gate).shape == (0, 40)
    assert gpu.gptq_gated_backward(dY[:0], X[:0], gate, gate).shape == (0, 96)
    assert gpu.gptq_linear_backward(dY[:0], *gate).shape == (0, 96)


@pytest.mark.gpu
@pytest.mark.parametrize("t,rows,n", [(20000, 260, 288), (17000, 520, 1056)])
def test_more_tokens_than_the_workspace_holds(gpu, t, rows, n):
    """Slices of 2^14 tokens, the last a short one: a sample of tokens of each."""
    for kind in TYPES:
        X, dY, gate, up, _ = make(t, rows, n, kind, "q4tp", 71)
        pick = torch.cat([torch.arange(20), torch.arange(16364, 16404), torch.arange(t - 20, t)])
        for got, (want, bound) in (
                (gpu.gptq_linear_backward(dY, *gate), layer.linear_backward(dY[pick], *gate, "q4tp")),
                (gpu.gptq_gated(X, gate, up), layer.gated(X[pick], gate, up, "q4tp", "silu", (None, None))),
                (gpu.gptq_gated_backward(dY, X, gate, up), layer.gated_backward(dY[pick], X[pick], gate, up, "q4tp", "silu", (None, None)))):
            ref.assert_within(got[pick.cuda()], want, bound, str(kind))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,rows,n", [(3, 200, 1056), (300, 2101, 2080), (1210, 2101, 2080)])
def test_streams_and_graphs(gpu, kind, t, rows, n):
    """Calls on a side stream, and captured ones with their workspaces inside, replayed on new inputs with eager work
    between: the eager results, bit for bit."""
    X, dY, gate, up, _ = make(t, rows, n, kind, "q4tp", 81)

    def step():
        y = gpu.gptq_gated(X, gate, up)
        return y, gpu.gptq_gated_backward(dY, X, gate, up), gpu.gptq_linear_backward(dY, *gate)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (gpu.gptq_gated(X, gate, up, stream=side), gpu.gptq_gated_backward(dY, X, gate, up, stream=side),
           gpu.gptq_linear_backward(dY, *gate, stream=side))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.cuda.graph(second):
        other = step()
    g = torch.Generator("cuda").manual_seed(1)
    for i in range(4):
        X.copy_(torch.randn(t, n, device="cuda", generator=g))
        dY.copy_(torch.randn(t, rows, device="cuda", generator=g))
        graph.replay()
        first = [z.clone() for z in out]
        second.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b, c in zip(first, other, want):
            assert torch.equal(a, c) and torch.equal(b, c), i


@pytest.mark.gpu
def test_workspaces_of_the_caller(gpu):
    t, rows, n = 1210, 2101, 2080
    X, dY, gate, up, _ = make(t, rows, n, torch.bfloat16, "q4tp", 91)
    w = [torch.full((k,), 255, dtype=torch.uint8, device="cuda") for k in
         (gpu.gated_workspace_size(t, rows, n), gpu.gated_workspace_size(t, rows, n, backward=True),
          gpu.linear_backward_workspace_size(t, rows, n))]
    assert torch.equal(gpu.gptq_gated(X, gate, up, workspace=w[0]), gpu.gptq_gated(X, gate, up))
    assert torch.equal(gpu.gptq_gated_backward(dY, X, gate, up, workspace=w[1]), gpu.gptq_gated_backward(dY, X, gate, up))
    assert torch.equal(gpu.gptq_linear_backward(dY, *gate, workspace=w[2]), gpu.gptq_linear_backward(dY, *gate))
    with pytest.raises(ValueError):
        gpu.gptq_gated(X, gate, up, workspace=w[0][:-256])
    with pytest.raises(gpu.GptqError):
        gpu.gptq_linear_backward(dY, *gate, out=dY[:, :2080])
