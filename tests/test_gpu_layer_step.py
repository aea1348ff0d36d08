"""The layer's further operators as they are used together: a decoder layer of this library's own fold and sweep with rotary
positions, a 4-bit cache whose tokens' attention is counted and which is cut back to a budget, and a gated block, over
prompts and then token by token, eagerly and from a captured graph; and the gradients back through its block."""
import math

import numpy as np
import pytest
import torch

import layer as ref2
import operands as ref

WIDTH, HEADS, GROUP, DIM, INNER = 256, 2, 2, 64, 416
QKV = (HEADS * GROUP + 2 * HEADS) * DIM
PART = 32


class Layer:
    """h + Wo attention(rotary(Wqkv h)), then h + Wd (silu(Wg h) * (Wu h)), with quantized weights."""

    def __init__(self, gpu, seed, pages=40, page=16):
        g = torch.Generator("cuda").manual_seed(seed)
        self.gpu = gpu
        X, Z = (torch.randn(1024, w, device="cuda", generator=g) for w in (WIDTH, INNER))
        rows = {"qkv": QKV, "o": WIDTH, "gate": INNER, "up": INNER}
        W = {k: torch.randn(r, WIDTH, device="cuda", generator=g) / math.sqrt(WIDTH) for k, r in rows.items()}
        down = torch.randn(WIDTH, INNER, device="cuda", generator=g) / math.sqrt(INNER)
        H, Hd = torch.zeros(WIDTH, WIDTH, device="cuda"), torch.zeros(INNER, INNER, device="cuda")
        gpu.gptq_gram_add(H, X)
        gpu.gptq_gram_add(Hd, Z)
        self.round = gpu.Round([dict(H=H, lam=0.01, members=list(W.values())), dict(H=Hd, lam=0.01, members=[down])])
        assert self.round.run() == 0
        pair = lambda i, k: (self.round.results[i]["members"][k][2], self.round.results[i]["members"][k][4])  # noqa: E731
        self.w = {k: pair(0, i) for i, k in enumerate(W)}
        self.w["down"] = pair(1, 0)
        self.freq, self.factor = gpu.rotary_frequencies(PART, scaling="ramp", stretch=2.0)
        self.cache = gpu.cache_alloc(pages, page, HEADS, DIM)
        self.score = gpu.score_alloc(self.cache)

    def __call__(self, h, position, table, length, start=None, parts=None):
        gpu, rows = self.gpu, h.shape[0]
        x = gpu.gptq_linear(h, *self.w["qkv"]).view(rows, -1, DIM)
        q, k, v = x.split([HEADS * GROUP, HEADS, HEADS], 1)
        before = x.clone() if parts is not None else None
        gpu.gptq_rotary(q, position, self.freq, K=k, factor=self.factor, out=(q, k))
        gpu.gptq_cache_write(self.cache, k, v, table, length, start)
        o, lse = gpu.gptq_cache_attention(self.cache, q, table, length, start, want_lse=True)
        old = self.score.clone() if parts is not None else None
        gpu.gptq_cache_score(self.cache, q, lse, self.score, table, length, start)
        y = gpu.gptq_linear(o.view(rows, -1), *self.w["o"], residual=h)
        z = self.round.gated(y, 0, 2, 3)
        out = gpu.gptq_linear(z, *self.w["down"], residual=y)
        if parts is not None:
            parts.update(before=before, q=q, k=k, v=v, o=o, lse=lse, old=old, y=y, z=z, out=out)
        return out

    def check(self, plain, h, position, table, length, start, parts):
        """Every link of a step against its definition on what the link before it gave."""
        tb, ln, st = (None if t is None else t.cpu().numpy() for t in (table, length, start))
        for got, was in ((parts["q"], parts["before"][:, :HEADS * GROUP]), (parts["k"], parts["before"][:, HEADS * GROUP:-HEADS])):
            want, bound = ref2.rotary(was, position, self.freq, "half", self.factor, False)
            ref.assert_within(got, want, bound, "rotary")
        plain.write(tb, ln, st, *(parts[n].double().cpu().numpy() for n in "kv"))
        for got, exp in zip(self.cache, plain.tensors("cuda")):
            assert torch.equal(got.view(torch.uint8), exp.view(torch.uint8))
        want, _, bound, _ = ref.attention(plain, parts["q"], tb, ln, st, 1 / math.sqrt(DIM), 0, 0)
        ref.assert_within(parts["o"], want, bound, "attention")
        want, bound, written = ref2.score(plain, parts["old"], parts["q"], parts["lse"], tb, ln, st, 1 / math.sqrt(DIM), 0, 0)
        score = self.score.double().cpu().numpy()
        ref.assert_within(score[written], want[written], bound[written], "score")
        assert np.array_equal(score[~written], parts["old"].double().cpu().numpy()[~written])
        want, bound = ref2.gated(parts["y"], self.w["gate"], self.w["up"], "q4tp", "silu", (None, None))
        ref.assert_within(parts["z"], want, bound, "gated")
        want, bound = ref.linear(parts["z"], *self.w["down"], "q4tp", None, "none", parts["y"])
        ref.assert_within(parts["out"], want, bound, "down")

    def evict(self, plain, table, length, keep, into=None):
        """Cut back, and the plain cache with it."""
        tb, ln = table.cpu().numpy(), length.cpu().numpy()
        want, index = ref2.evict(plain, self.score.cpu().numpy(), tb, ln, keep, 2, 5)
        left, kept = self.gpu.gptq_cache_evict(self.cache, table, length, self.score, keep, 2, 5, into=into)
        assert np.array_equal(left.cpu().numpy(), want) and np.array_equal(kept.cpu().numpy(), index)
        dest = tb if into is None else into.cpu().numpy()
        for plane in (plain.k, plain.v, plain.ks, plain.vs):
            moved = plane.copy()
            for b in range(tb.shape[0]):
                for h in range(HEADS):
                    for j in range(want[b]):
                        (tp, to), (fp, fo) = plain.place(dest, b, j), plain.place(tb, b, int(index[b, h, j]))
                        moved[tp, h, to] = plane[fp, h, fo]
            plane[:] = moved
        return left


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
def test_prompts_tokens_and_evictions(gpu, kind):
    """Prompts of three sequences, then tokens of two, cut back to a budget in place and to other pages on the way, the
    text's positions going on."""
    layer, plain = Layer(gpu, 1), ref.Cache(40, 16, HEADS, DIM)
    for s in (plain.k, plain.v):
        s[:] = layer.cache.k.cpu().numpy()
    lengths = [37, 5, 64]
    g = torch.Generator().manual_seed(2)
    table = torch.randperm(40, generator=torch.Generator().manual_seed(3))[:15].view(3, 5).to(torch.int32).cuda()
    free = torch.tensor(sorted(set(range(40)) - set(table.flatten().tolist())), dtype=torch.int32, device="cuda")
    h, start = torch.randn(106, WIDTH, generator=g).to(kind).cuda(), i32(0, 37, 42, 106)
    position, parts = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths]).cuda(), {}
    layer(h, position, table, i32(*lengths), start, parts)
    layer.check(plain, h, position, table, i32(*lengths), start, parts)
    two, cached, at = table[[0, 2]].contiguous(), i32(37, 64), i32(37, 64)
    for i in range(9):
        if i == 3:
            cached = layer.evict(plain, two, cached, 32)
        if i == 6:
            into = free[:10].view(2, 5).contiguous()
            cached, two = layer.evict(plain, two, cached, 20, into), into
        h = torch.randn(2, WIDTH, generator=g).to(kind).cuda()
        cached = cached + 1
        layer(h, at, two, cached, None, parts)
        layer.check(plain, h, at, two, cached, None, parts)
        at = at + 1


@pytest.mark.gpu
def test_captured_steps(gpu):
    """A step and the eviction behind it, captured once and replayed while the sequences grow, with eager work between."""
    a, b = Layer(gpu, 5), Layer(gpu, 5)
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 12).contiguous()
    h = torch.zeros(2, WIDTH, dtype=torch.bfloat16, device="cuda")
    length, position = i32(1, 40), i32(0, 39)

    def step(l):
        y = l(h, position, table, length)
        left, kept = gpu.gptq_cache_evict(l.cache, table, length, l.score, 44, 2, 5)
        return y, left, kept

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    torch.cuda.current_stream().wait_stream(side)
    for t in (*a.cache, a.score):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a)
    g = torch.Generator("cuda").manual_seed(6)
    now = [1, 40]
    for i in range(20):
        h.copy_(torch.randn(2, WIDTH, device="cuda", generator=g))
        length.copy_(i32(*now))
        position.copy_(i32(i, 39 + i))
        graph.replay()
        got = [t.clone() for t in out]
        want = step(b)
        torch.cuda.synchronize()
        for p, q in zip((*got, a.score, *a.cache), (*want, b.score, *b.cache)):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), i
        now = [n + 1 for n in got[1].tolist()]
    assert now[1] == 45


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
def test_gradients_through_the_block(gpu, kind):
    """dL/dy of y + Wd (silu(Wg y) * (Wu y)), link by link, and rotary's transpose of a projection's gradient."""
    layer = Layer(gpu, 9)
    g = torch.Generator().manual_seed(4)
    y, d = (torch.randn(50, WIDTH, generator=g).to(kind).cuda() for _ in range(2))
    dz = gpu.gptq_linear_backward(d, *layer.w["down"])
    want, bound = ref2.linear_backward(d, *layer.w["down"], "q4tp")
    ref.assert_within(dz, want, bound, "down")
    dy = gpu.gptq_gated_backward(dz, y, layer.w["gate"], layer.w["up"])
    want, bound = ref2.gated_backward(dz, y, layer.w["gate"], layer.w["up"], "q4tp", "silu", (None, None))
    ref.assert_within(dy, want, bound, "block")
    dq = torch.randn(50, HEADS, DIM, generator=g).to(kind).cuda()
    p = torch.arange(50, dtype=torch.int32, device="cuda")
    back = gpu.gptq_rotary(dq, p, layer.freq, factor=layer.factor, backward=True)
    want, bound = ref2.rotary(dq, p, layer.freq, "half", layer.factor, True)
    ref.assert_within(back, want, bound, "rotary")


@pytest.mark.gpu
def test_two_streams_at_once(gpu):
    """Two layers' steps and gradients on two streams: what each gives alone."""
    layers = [Layer(gpu, s) for s in (7, 8)]
    table, ln, st = torch.arange(24, dtype=torch.int32, device="cuda").view(1, 24), i32(300), i32(0, 300)
    position = torch.arange(300, dtype=torch.int32, device="cuda")
    h = [torch.randn(300, WIDTH, device="cuda", generator=torch.Generator("cuda").manual_seed(s)).to(torch.bfloat16) for s in (1, 2)]

    def step(l, x):
        y = l(x, position, table, ln, st)
        dz = gpu.gptq_linear_backward(x, *l.w["down"])
        return y, dz, gpu.gptq_gated_backward(dz, y, l.w["gate"], l.w["up"]), l.score.clone()

    want = [step(l, x) for l, x in zip(layers, h)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        got = []
        for l, x, s in zip(layers, h, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step(l, x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for p, q in zip(a, b):
                assert torch.equal(p, q)
