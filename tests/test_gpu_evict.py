"""The cache's scores and eviction against their definitions: types, head layouts, pages, lengths from none on, windows,
absent pages, old scores, ties, values that are not finite, moves in place and to other pages."""
import numpy as np
import pytest
import torch

import layer
import operands as ref

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def filled(pages, page, heads, dim, seed):
    """A cache with random codes -7..7 and scales of 5 bits."""
    c, r = ref.Cache(pages, page, heads, dim), np.random.RandomState(seed)
    for plane in (c.k, c.v):
        plane[:] = r.randint(1, 16, plane.shape) | r.randint(1, 16, plane.shape) << 4
    for s in (c.ks, c.vs):
        s[:] = np.ldexp(r.randint(16, 32, s.shape), r.randint(-8, -5, s.shape))
    return c


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def run_score(gpu, c, kind, table, length, start, rows, group, window=0, sinks=0, scale=None, seed=0, in_place=False, q=None):
    g = torch.Generator().manual_seed(seed)
    Q = torch.randn(rows, c.heads * group, c.dim, generator=g).to(kind).cuda() if q is None else q
    planes = c.tensors("cuda")
    t, n, s = i32(table), i32(length), None if start is None else i32(start)
    scale = c.dim ** -0.5 if scale is None else scale
    _, lse = gpu.gptq_cache_attention(planes, Q, t, n, s, scale=scale, window=window, sinks=sinks, want_lse=True)
    old = torch.rand(c.pages, c.heads, c.page, generator=g).cuda()
    want, bound, written = layer.score(c, old, Q, lse, table, length, start, scale, window, sinks)
    out = old.clone() if in_place else torch.full_like(old, -3.0)
    got = gpu.gptq_cache_score(planes, Q, lse, out if in_place else old, t, n, s, scale=scale, window=window, sinks=sinks,
                               out=None if in_place else out)
    assert got is out
    out = out.double().cpu().numpy()
    ref.assert_within(out[written], want[written], bound[written], "score")
    assert (out[~written] == (old.double().cpu().numpy()[~written] if in_place else -3.0)).all()
    return out, lse, Q


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 3, 1), (128, 32, 2, 5), (256, 16, 1, 16), (128, 48, 1, 33)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3), (1, 0), (64, 100)])
def test_scores(gpu, kind, dim, page, heads, group, window, sinks):
    """Ragged sequences: one token, whole prompts, drafts over a long past, an empty one between."""
    rows = [1, 70, 5, 0, 33]
    length = np.array([1, 70, 300, 0, 200])
    c = filled(60, page, heads, dim, dim + group)
    width = -(-300 // page)
    table = np.full((5, width), -1, np.int32)
    perm = np.random.RandomState(1).permutation(60)
    for b, n in enumerate(length):
        k = -(-n // page)
        table[b, :k], perm = perm[:k], perm[k:]
    start = np.concatenate([[0], np.cumsum(rows)])
    for in_place in (False, True):
        run_score(gpu, c, kind, table, length, start, 109, group, window, sinks, seed=window, in_place=in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
def test_single_rows(gpu, kind):
    length = np.array([1, 15, 16, 17, 255, 256, 257, 600])
    c = filled(80, 16, 2, 128, 3)
    table = np.random.RandomState(2).permutation(80)[:8 * 10].reshape(8, 10)
    table = np.concatenate([table, np.full((8, 30), 999)], 1).astype(np.int32)  # pages that are not there
    run_score(gpu, c, kind, table, length, None, 8, 4, seed=1)
    run_score(gpu, c, kind, table, length, None, 8, 8, window=100, sinks=2, seed=2, scale=-0.2)


@pytest.mark.gpu
def test_scores_of_rows_before_the_first_token(gpu):
    """More rows than tokens, lengths past the table, negative ones, rows behind the last sequence."""
    c = filled(12, 16, 2, 64, 4)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    run_score(gpu, c, torch.bfloat16, table, np.array([3, 500, -7]), np.array([0, 9, 12, 14]), 20, 3, seed=3)


@pytest.mark.gpu
def test_hidden_values_that_are_not_finite(gpu):
    """NaN scales of tokens behind a sequence's end or out of its window, and old scores where rows are new."""
    c = filled(8, 16, 1, 64, 5)
    table = np.array([[3, 5, 1, 7]], np.int32)
    length, start = np.array([50]), np.array([0, 4])
    a, lse, Q = run_score(gpu, c, torch.bfloat16, table, length, start, 4, 2, window=8, sinks=1, seed=4)
    for t in list(range(1, 38)) + list(range(50, 64)):
        at = c.place(table, 0, t)
        c.ks[at[0], :, at[1]] = np.nan
    planes = c.tensors("cuda")
    old = torch.full((8, 1, 16), float("nan"), device="cuda")
    for t in range(46):
        old[table[0, t // 16], 0, t % 16] = 0.5
    out = gpu.gptq_cache_score(planes, Q, lse, old, i32(table), i32(length), i32(start), window=8, sinks=1, out=torch.zeros_like(old))
    got = [float(out[table[0, t // 16], 0, t % 16]) for t in range(50)]
    assert np.isfinite(got).all() and got[1:38] == [0.5] * 37


@pytest.mark.gpu
def test_long_scores(gpu):
    """A sequence far longer than a workgroup's piece, weights that add up to the number of rows and heads."""
    pages, page, heads, group = 1300, 16, 2, 4
    c = filled(4, page, heads, 128, 6)
    planes = [p.repeat(325, 1, 1, 1).contiguous() for p in c.tensors("cuda")]
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(1, -1).cuda()
    n = 20793
    Q = torch.randn(100, heads * group, 128, generator=torch.Generator().manual_seed(2)).cuda()
    length, start = i32([n]), i32([0, 100])
    _, lse = gpu.gptq_cache_attention(planes, Q, table, length, start, want_lse=True)
    out = gpu.gptq_cache_score(planes, Q, lse, torch.zeros(pages, heads, page, device="cuda"), table, length, start)
    assert torch.equal(out, gpu.gptq_cache_score(planes, Q, lse, torch.zeros_like(out), table, length, start))
    total = out.double().sum((0, 2))
    assert float((total - 100 * group).abs().max()) < 100 * group * 2.0 ** -15
    assert int((out[table[0, -1].long()] != 0).sum()) == heads * (n % page)


def run_evict(gpu, c, score, table, length, keep, sinks, recent, into=None):
    want, index = layer.evict(c, score, table, length, keep, sinks, recent)
    planes, z = c.tensors("cuda"), torch.from_numpy(score.copy()).cuda()
    before = [p.clone().cpu() for p in planes] + [z.clone().cpu()]
    left, kept = gpu.gptq_cache_evict(planes, i32(table), i32(length), z, keep, sinks, recent, into=None if into is None else i32(into))
    assert np.array_equal(left.cpu().numpy(), want) and np.array_equal(kept.cpu().numpy(), index)
    # Every place of the planes: moved, or as it was.
    dest = table if into is None else into
    wanted = [p.clone() for p in before]
    zero = [0x88, 0x88, 0.0, 0.0, 0.0]
    for b in range(table.shape[0]):
        for h in range(c.heads):
            for j in range(want[b]):
                to, at = c.place(dest, b, j), c.place(table, b, int(index[b, h, j]))
                if to is None or (into is None and index[b, h, j] == j):
                    continue
                for w, old, fill in zip(wanted, before, zero):
                    w[to[0], h, to[1]] = fill if at is None else old[at[0], h, at[1]]
    for got, w in zip((*planes, z), wanted):
        assert torch.equal(got.cpu().view(torch.uint8), w.contiguous().view(torch.uint8))


def scores(c, seed, kind="spread"):
    r = np.random.RandomState(seed)
    z = np.exp(2 * r.randn(c.pages, c.heads, c.page) - 4).astype(np.float32)
    if kind == "ties":
        z = np.round(z * 4).astype(np.float32) / 4
    if kind == "wild":
        z *= np.where(r.rand(*z.shape) < 0.5, -1, 1)
        z[r.rand(*z.shape) < 0.05] = np.nan
        z[r.rand(*z.shape) < 0.05] = np.inf
        z[r.rand(*z.shape) < 0.05] = -np.inf
        z[r.rand(*z.shape) < 0.1] = 0.0
        z[r.rand(*z.shape) < 0.1] = -0.0
    return z.astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 3), (128, 48, 2), (256, 16, 1)])
@pytest.mark.parametrize("kind", ["spread", "ties", "wild"])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (40, 0, 0), (64, 4, 16), (64, 4, 60), (65, 65, 0), (500, 3, 7)])
def test_eviction(gpu, dim, page, heads, kind, keep, sinks, recent):
    """Sequences shorter than the budget, of its length, one over, far over, empty; in place and to other pages."""
    length = np.array([0, 1, 64, 65, 300, 129])
    k = -(-length // page)
    c = filled(int(k.sum()) + 80, page, heads, dim, dim)
    perm = np.random.RandomState(5).permutation(c.pages)
    table = np.full((6, int(k.max())), -1, np.int32)
    for b in range(6):
        table[b, :k[b]], perm = perm[:k[b]], perm[k[b]:]
    z = scores(c, keep, kind)
    run_evict(gpu, c, z, table, length, keep, sinks, recent)
    wide = -(-min(keep, 300) // page)
    into = np.resize(perm, 6 * wide).reshape(6, wide).astype(np.int32) if 6 * wide <= len(perm) else np.full((6, wide), -1, np.int32)
    if 6 * wide > len(perm):
        into[4] = perm[:wide]
    run_evict(gpu, c, z, table, length, keep, sinks, recent, into)


@pytest.mark.gpu
@pytest.mark.parametrize("n,keep", [(1024, 1023), (2049, 1024), (9000, 8900), (9000, 100), (20000, 300)])
def test_long_evictions(gpu, n, keep):
    """Sequences of several turns, and of more tokens than a workgroup keeps the keys of."""
    c = filled(-(-n // 128) + 3, 128, 2, 64, n)
    table = np.random.RandomState(n).permutation(c.pages)[:-(-n // 128)].reshape(1, -1).astype(np.int32)
    for kind in ("spread", "ties"):
        run_evict(gpu, c, scores(c, n, kind), table, np.array([n]), keep, 4, keep // 3)


@pytest.mark.gpu
def test_absent_pages(gpu):
    """Tokens without a place go first, are zeros where they are protected, and places that are not there drop what
    would go to them; lengths past the table count as the table's."""
    c = filled(10, 16, 2, 64, 9)
    table = np.array([[0, 99, 2, 3], [4, -1, 6, 1 << 30]], np.int32)
    z = scores(c, 3)
    run_evict(gpu, c, z, table, np.array([60, 64]), 30, 2, 5)
    run_evict(gpu, c, z, table, np.array([1000, -4]), 30, 20, 5)
    run_evict(gpu, c, z, table, np.array([64, 64]), 34, 20, 5, np.array([[7, 77, 8], [-1, 9, 1]], np.int32)[:, :2])


@pytest.mark.gpu
def test_evictions_again(gpu):
    """The same call twice gives the same; a captured one replays with new lengths and scores."""
    c = filled(40, 16, 2, 128, 11)
    table = np.arange(40, dtype=np.int32).reshape(2, 20)
    planes, z = c.tensors("cuda"), torch.from_numpy(scores(c, 1)).cuda()
    t, length = i32(table[:, :10]), i32([150, 160])
    into = i32(table[:, 10:15])
    gpu.gptq_cache_evict(planes, t, length, z, 70, 2, 8, into=into)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        left, kept = gpu.gptq_cache_evict(planes, t, length, z, 70, 2, 8, into=into)
    for i in range(4):
        z.copy_(torch.from_numpy(scores(c, i + 5, "ties")))
        length.copy_(i32([60 + 30 * i, 160 - 7 * i]))
        graph.replay()
        got = [x.clone() for x in (left, kept, z, *planes)]
        other = gpu.gptq_cache_evict(planes, t, length, z, 70, 2, 8, into=into)
        for a, b in zip(got, (*other, z, *planes)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
        want, index = layer.evict(c, z.cpu().numpy(), table[:, :10], length.cpu().numpy(), 70, 2, 8)
        assert np.array_equal(got[0].cpu().numpy(), want) and np.array_equal(got[1].cpu().numpy(), index)
