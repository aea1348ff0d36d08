"""The operators on quantized operands as they are used together: a decoder layer whose projections are
codes of this library's own fold and sweep, its keys and values in a 4-bit cache, run over a prompt
and then token by token, eagerly and from a captured graph; and two layers' steps on two streams."""
import math

import pytest
import torch

import operands as ref

WIDTH, HEADS, GROUP, DIM = 256, 2, 2, 64
QKV = (HEADS * GROUP + 2 * HEADS) * DIM


class Layer:
    """h + Wo attention(Wqkv h) with quantized weights and cache."""

    def __init__(self, gpu, seed, pages=24, page=16):
        g = torch.Generator("cuda").manual_seed(seed)
        self.gpu = gpu
        X = torch.randn(1024, WIDTH, device="cuda", generator=g)
        W = [torch.randn(r, WIDTH, device="cuda", generator=g) / math.sqrt(WIDTH) for r in (QKV, WIDTH)]
        H = torch.zeros(WIDTH, WIDTH, device="cuda")
        gpu.gptq_gram_add(H, X)
        self.round = gpu.Round([dict(H=H, lam=0.01, members=[W[0], (W[1], "q4tp")])])
        assert self.round.run() == 0
        self.bias = torch.randn(QKV, device="cuda", generator=g) * 0.1
        self.cache = gpu.cache_alloc(pages, page, HEADS, DIM)

    def __call__(self, h, table, length, start=None, parts=None):
        gpu = self.gpu
        x = self.round.linear(h, 0, 0, bias=self.bias).view(h.shape[0], -1, DIM)
        q, k, v = x.split([HEADS * GROUP, HEADS, HEADS], 1)
        gpu.gptq_cache_write(self.cache, k, v, table, length, start)
        o = gpu.gptq_cache_attention(self.cache, q, table, length, start)
        y = self.round.linear(o.view(h.shape[0], -1), 0, 1, residual=h)
        if parts is not None:
            parts.update(x=x, q=q, k=k, v=v, o=o, y=y)
        return y

    def check(self, plain, h, table, length, start, parts):
        """Every link of a step against its definition on what the link before it gave, at that
        link's own bounds; ``plain`` is the cache so far, on the CPU."""
        r = self.round.results[0]["members"]
        want, bound = ref.linear(h, r[0][2], r[0][4], "q4tp", self.bias, "none", None)
        ref.assert_within(parts["x"].reshape(h.shape[0], -1), want, bound, "projection")
        tb, ln, st = (None if t is None else t.cpu().numpy() for t in (table, length, start))
        plain.write(tb, ln, st, *(parts[n].double().cpu().numpy() for n in "kv"))
        for got, exp in zip(self.cache, plain.tensors("cuda")):
            assert torch.equal(got.view(torch.uint8), exp.view(torch.uint8))
        want, _, bound, _ = ref.attention(plain, parts["q"], tb, ln, st, 1 / math.sqrt(DIM), 0, 0)
        ref.assert_within(parts["o"], want, bound, "attention")
        want, bound = ref.linear(parts["o"].reshape(h.shape[0], -1), r[1][2], r[1][4], "q4tp", None, "none", h)
        ref.assert_within(parts["y"], want, bound, "output")


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
def test_prompt_then_tokens(gpu, kind):
    """Prompts of three sequences at once, then some tokens of two of them, one at a time."""
    layer, plain = Layer(gpu, 1), ref.Cache(24, 16, HEADS, DIM)
    for s in (plain.k, plain.v):
        s[:] = layer.cache.k.cpu().numpy()
    lengths = [37, 5, 64]
    g = torch.Generator().manual_seed(2)
    table = torch.randperm(24, generator=torch.Generator().manual_seed(3))[:15].view(3, 5).to(torch.int32).cuda()
    parts = {}
    h = torch.randn(sum(lengths), WIDTH, generator=g).to(kind).cuda()
    start = i32(0, 37, 42, 106)
    layer(h, table, i32(*lengths), start, parts)
    layer.check(plain, h, table, i32(*lengths), start, parts)
    two = table[[0, 2]].contiguous()
    for i in range(1, 12):
        h = torch.randn(2, WIDTH, generator=g).to(kind).cuda()
        length = i32(37 + i, 64 + i)
        layer(h, two, length, None, parts)
        layer.check(plain, h, two, length, None, parts)


@pytest.mark.gpu
def test_captured_steps(gpu):
    """A step captured once and replayed while the sequences grow, with eager work between."""
    a, b = Layer(gpu, 5), Layer(gpu, 5)
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 12).contiguous()
    h = torch.zeros(2, WIDTH, dtype=torch.bfloat16, device="cuda")
    length = i32(1, 40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a(h, table, length)
    torch.cuda.current_stream().wait_stream(side)
    for t in a.cache:
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = a(h, table, length)
    g = torch.Generator("cuda").manual_seed(6)
    for i in range(20):
        h.copy_(torch.randn(2, WIDTH, device="cuda", generator=g))
        length.copy_(i32(i + 1, 40 + i))
        graph.replay()
        got = y.clone()
        want = b(h, table, length)
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
        for p, q in zip(a.cache, b.cache):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.gpu
def test_two_streams_at_once(gpu):
    layers = [Layer(gpu, s) for s in (7, 8)]
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(1, 24)
    h = [torch.randn(300, WIDTH, device="cuda", generator=torch.Generator("cuda").manual_seed(s)).to(torch.bfloat16) for s in (1, 2)]
    ln, st = i32(300), i32(0, 300)
    want = [l(x, table, ln, st) for l, x in zip(layers, h)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        got = []
        for l, x, s in zip(layers, h, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(l(x, table, ln, st))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
