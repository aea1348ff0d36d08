"""The product with the codes (gptq_linear) against its definition in 64 bits: types, codecs, sizes
from one token and one row up, ragged quads of groups, epilogues, strides, extreme scales, values that
are not finite, other streams and captured graphs."""
import pytest
import torch

import operands as ref

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(t, rows, n, kind, codec, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(t, n, generator=g) * torch.where(torch.rand(n, generator=g) < 0.03, 20.0, 1.0)
    codes = torch.randint(0, 256, (rows, n // (2 if codec == "q4tp" else 4)), generator=g, dtype=torch.uint8)
    scale = torch.exp2(torch.randn(rows, n // 32, generator=g) * spread - 6.0)
    bias = torch.randn(rows, generator=g)
    residual = torch.randn(t, rows, generator=g).to(kind)
    return X.to(kind).cuda(), codes.cuda(), scale.cuda(), bias.cuda(), residual.cuda()


def check(gpu, X, codes, scale, codec, bias=None, act="none", residual=None, what="", **kw):
    y = gpu.gptq_linear(X, codes, scale, codec, bias, act, residual, **kw)
    want, bound = ref.linear(X, codes, scale, codec, bias, act, residual)
    assert y.dtype == X.dtype
    ref.assert_within(y, want, bound, what)
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", [(1, 1, 32), (1, 16, 64), (2, 17, 96), (15, 33, 128), (16, 64, 160), (17, 31, 1024),
                                      (31, 100, 480), (33, 7, 2080), (64, 48, 4128), (65, 200, 256), (127, 129, 544),
                                      (128, 257, 64), (200, 130, 992), (300, 515, 1504), (513, 260, 320), (250, 555, 544),
                                      (400, 1030, 96), (97, 1411, 2080)])
def test_sizes(gpu, kind, codec, t, rows, n):
    X, codes, scale, bias, residual = make(t, rows, n, kind, codec, t * 7 + rows)
    check(gpu, X, codes, scale, codec, what="plain")
    check(gpu, X, codes, scale, codec, bias, "gelu", residual, what="gelu, all")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", [(40, 520, 2176), (24, 8200, 4224), (9, 8200, 4128), (1, 20000, 2048), (130, 8300, 4128),
                                      (70, 1030, 1440), (20, 40000, 1024), (3, 300000, 128), (600, 9000, 128), (250, 1030, 1440),
                                      (90, 2050, 2080)])
def test_pieces_of_k(gpu, kind, codec, t, rows, n):
    """Sizes whose sums are cut along K or whose rows are many: every piece, uneven ones and the last
    quads of groups among them.  A sample of rows, which the others share no sums with."""
    X, codes, scale, bias, residual = make(t, rows, n, kind, codec, rows)
    y = gpu.gptq_linear(X, codes, scale, codec, bias, "silu", residual)
    pick = torch.cat([torch.arange(0, 40), torch.arange(rows - 40, rows), torch.randint(0, rows, (200,))]).cuda()
    want, bound = ref.linear(X, codes[pick], scale[pick], codec, bias[pick], "silu", residual[:, pick])
    ref.assert_within(y[:, pick], want, bound, "pieces")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n,act,pad", [(300, 8301, 2080, "gelu", 0), (2100, 1030, 2400, "none", 2), (513, 20000, 544, "silu", 0),
                                              (4100, 264, 4960, "relu", 8), (777, 2056, 4128, "gelu_tanh", 0)])
def test_large_products(gpu, kind, codec, t, rows, n, act, pad):
    """Products large enough for decoded weights: rows that keep Y aligned and that do not, X and Y padded, the
    residual in place, scales octaves apart, a NaN and an infinity that stay in their tokens."""
    X, codes, scale, bias, residual = make(t, rows, n, kind, codec, t)
    low, high = (-10, 4) if kind is torch.float16 else (-50, 50)
    scale *= torch.exp2(torch.linspace(low, high, rows, device="cuda").round())[:, None]
    scale[5] = 0.0
    wide = torch.full((t, n + 32), float("nan"), dtype=kind, device="cuda")
    wide[:, 16:16 + n] = X * 0.01
    x = wide[:, 16:16 + n]
    keep = torch.full((t, rows + pad), 3.0, dtype=kind, device="cuda")
    keep[:, :rows] = residual
    y = keep[:, :rows]
    pick = torch.cat([torch.arange(0, 70), torch.arange(rows - 70, rows), torch.randint(0, rows, (60,))]).cuda()
    want, bound = ref.linear(x, codes[pick], scale[pick], codec, bias[pick], act, residual[:, pick])
    gpu.gptq_linear(x, codes, scale, codec, bias, act, y, out=y)
    top = 65504.0 if kind is torch.float16 else 3.0e38
    fine = want.abs().amax(0) < top / 2
    assert fine.sum() > 120
    ref.assert_within(y[:, pick][:, fine.cuda()], want[:, fine], bound[:, fine], "large")
    assert (keep[:, rows:] == 3).all()
    clean = gpu.gptq_linear(x, codes, scale, codec, bias, act)
    x[2, 7], x[t - 3, n - 1] = float("nan"), float("inf")
    bad = gpu.gptq_linear(x, codes, scale, codec, bias, act)
    others = [i for i in range(t) if i not in (2, t - 3)]
    assert torch.equal(bad[others], clean[others]) and not torch.isfinite(bad[2]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("t", [2, 60, 300])
def test_far_rows(gpu, t):
    """Codes and decoded weights whose bytes pass 2^32, by their last rows."""
    rows, n = 540000, 16384
    g = torch.Generator("cuda").manual_seed(t)
    X = torch.randn(t, n, device="cuda", generator=g, dtype=torch.bfloat16)
    codes = torch.randint(0, 256, (rows, n // 2), device="cuda", dtype=torch.uint8, generator=g)
    scale = torch.rand(rows, n // 32, device="cuda", generator=g) * 0.01
    y = gpu.gptq_linear(X, codes, scale)
    pick = torch.cat([torch.arange(20), torch.arange(rows // 2, rows // 2 + 20), torch.arange(rows - 40, rows)]).cuda()
    want, bound = ref.linear(X, codes[pick], scale[pick], "q4tp", None, "none", None)
    ref.assert_within(y[:, pick], want, bound, "far")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t", [3, 260, 2100])
def test_epilogues(gpu, act, kind, t):
    X, codes, scale, bias, residual = make(t, 130, 288, kind, "q4tp", 5)
    for b in (None, bias):
        for r in (None, residual):
            check(gpu, X, codes, scale, "q4tp", b, act, r, what=f"{act} {b is not None} {r is not None}")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t", [1, 5, 300, 1500])
def test_strides_and_residual_in_place(gpu, kind, t):
    """Padded rows of X, of the residual and of Y, whose own columns alone are written."""
    rows, n = 75, 224
    X, codes, scale, bias, residual = make(t, rows, n, kind, "q4tp", 9)
    wide = torch.full((t, n + 64), float("nan"), dtype=kind, device="cuda")
    wide[:, 32:32 + n] = X
    keep = torch.full((t, rows + 9), 3.0, dtype=kind, device="cuda")
    keep[:, 4:4 + rows] = residual
    y = keep[:, 4:4 + rows]
    want, bound = ref.linear(X, codes, scale, "q4tp", bias, "silu", residual)
    out = gpu.gptq_linear(wide[:, 32:32 + n], codes, scale, "q4tp", bias, "silu", y, out=y)
    assert out is y
    ref.assert_within(y, want, bound, "in place")
    assert (keep[:, :4] == 3).all() and (keep[:, 4 + rows:] == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t", [4, 280, 2100])
def test_scales_of_any_size(gpu, kind, t):
    """Rows whose scales lie many octaves apart, far from 1, or are zero."""
    X, codes, scale, _, _ = make(t, 64, 256, kind, "q4tp", 11, spread=3.0)
    low, high = (-24, 6) if kind is torch.float16 else (-60, 60)
    scale *= torch.exp2(torch.linspace(low, high, 64, device="cuda").round())[:, None]
    scale[5] = 0.0
    scale[6, ::2] = 0.0
    X = X * 0.01
    want, bound = ref.linear(X, codes, scale, "q4tp", None, "none", None)
    y = gpu.gptq_linear(X, codes, scale)
    top = 65504.0 if kind is torch.float16 else 3.0e38
    fine = want.abs().amax(0) < top / 2
    ref.assert_within(y[:, fine.cuda()], want[:, fine], bound[:, fine], "scales")
    assert fine.sum() > 48 and (y[:, 5] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t", [16, 290, 1400])
def test_values_not_finite_stay_in_their_token(gpu, kind, t):
    X, codes, scale, bias, _ = make(t, 70, 128, kind, "q4tp", 13)
    clean = gpu.gptq_linear(X, codes, scale, bias=bias)
    bad = X.clone()
    bad[2, 7] = float("nan")
    bad[t - 3, 127] = float("inf")
    y = gpu.gptq_linear(bad, codes, scale, bias=bias)
    others = [i for i in range(t) if i not in (2, t - 3)]
    assert torch.equal(y[others], clean[others])
    assert not torch.isfinite(y[2]).any()
    assert (~torch.isfinite(y[t - 3])).float().mean() > 0.9  # a code of value 0 meets inf in at most a few rows


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 40, 250, 700])
def test_same_bits_every_time_and_on_any_stream(gpu, t):
    X, codes, scale, bias, residual = make(t, 300, 2048, torch.bfloat16, "q4tp", 17)
    y = gpu.gptq_linear(X, codes, scale, "q4tp", bias, "gelu", residual)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = gpu.gptq_linear(X, codes, scale, "q4tp", bias, "gelu", residual, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, z)
    need = gpu.linear_workspace_size(t, 300, 2048)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    assert torch.equal(y, gpu.gptq_linear(X, codes, scale, "q4tp", bias, "gelu", residual, workspace=ws))


@pytest.mark.gpu
def test_empty_and_wrong_arguments(gpu):
    X, codes, scale, bias, residual = make(4, 40, 64, torch.bfloat16, "q4tp", 19)
    assert gpu.gptq_linear(X[:0], codes, scale).shape == (0, 40)
    for bad in (dict(X=X.double()), dict(codes=codes[:, :8]), dict(scale=scale[:, :1]), dict(codec="q8"), dict(act="tanh"),
                dict(bias=bias[:3]), dict(residual=residual.float()), dict(residual=residual[:, :5]), dict(X=X.t()),
                dict(codes=codes.cpu()), dict(out=torch.empty(4, 41, dtype=torch.bfloat16, device="cuda"))):
        kw = dict(X=X, codes=codes, scale=scale)
        kw.update(bad)
        with pytest.raises(ValueError):
            gpu.gptq_linear(**kw)
    big = torch.zeros(4, 72, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu.GptqError):
        gpu.gptq_linear(big[:, 1:65], codes, scale)  # rows not 16-byte aligned


@pytest.mark.gpu
def test_of_a_round(gpu):
    """A round's members multiply by their own codes: against the weights those codes stand for."""
    import workloads
    H, W, lam = workloads.make("fixture", device="cuda:0")
    r = gpu.Round([dict(H=H, lam=lam, members=[W, (W.flip(0).contiguous(), "q2tp")])])
    assert r.run() == 0
    X = torch.randn(9, 160, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    for m, codec in ((0, "q4tp"), (1, "q2tp")):
        _, _, codes, _, scale = r.results[0]["members"][m]
        y = r.linear(X, 0, m, act="relu")
        want, bound = ref.linear(X, codes, scale, codec, None, "relu", None)
        ref.assert_within(y, want, bound, codec)
        near = torch.relu(X @ (W if m == 0 else W.flip(0)).t())
        assert (y - near).norm() < (0.25 if m == 0 else 0.9) * near.norm()


def captured(gpu, sizes):
    """One graph of a call of each size after the other: the calls as functions, X's, Y's and the graph."""
    calls, xs, ys = [], [], []
    for t, rows, n in sizes:
        X, codes, scale, bias, residual = make(t, rows, n, torch.bfloat16, "q4tp", t + n)
        xs.append(X)
        calls.append(lambda X=X, c=codes, s=scale, b=bias, r=residual: gpu.gptq_linear(X, c, s, "q4tp", b, "silu", r))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for call in calls:
            call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = [call() for call in calls]
    return calls, xs, ys, graph


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[(9, 8200, 4128)], [(40, 520, 2176), (24, 4200, 4224)], [(1100, 8205, 608)], [(2600, 6213, 800), (9, 8200, 4128)],
                                   [(1000, 2056, 4128), (777, 2056, 4128), (1100, 8216, 608)]])
def test_captured_graphs(gpu, sizes):
    """Calls with workspaces (pieces of K, decoded weights, cut tiles), several sharing a graph's memory: each
    replay on new inputs gives an eager call's bits, with eager calls and other work between replays."""
    calls, xs, ys, graph = captured(gpu, sizes)
    g = torch.Generator("cuda").manual_seed(3)
    for i in range(6):
        for X in xs:
            X.copy_(torch.randn(X.shape, device="cuda", generator=g) * (i + 1))
        graph.replay()
        got = [y.clone() for y in ys]
        want = [call() for call in calls]
        junk = [torch.randn(1 << 20, device="cuda", generator=g) for _ in range(3)]
        if i % 2:
            torch.cuda.synchronize()
            del junk
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


@pytest.mark.gpu
def test_two_graphs_of_one_pool(gpu):
    """Two graphs whose workspaces come from one pool, replayed in turn, keep their own outputs."""
    first, second = captured(gpu, [(2600, 6213, 800)]), captured(gpu, [(9, 8200, 4128)])
    pool = torch.cuda.graph_pool_handle()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph, c in zip(graphs, (first, second)):
        with torch.cuda.graph(graph, pool=pool):
            outs.append(c[0][0]())
    want = [c[0][0]() for c in (first, second)]
    for _ in range(4):
        for graph, out, w in zip(graphs, outs, want):
            graph.replay()
            assert torch.equal(out, w)
        torch.cuda.synchronize()
