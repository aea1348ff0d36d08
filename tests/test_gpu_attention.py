"""Attention over the 4-bit cache (gptq_cache_attention) against its definition in 64 bits: types,
head sizes and groups, lengths from zero and one up, rows from one to many, windows with sinks, pages that
end inside a block, absent and poisoned pages, rows that see nothing, rows behind the last sequence."""
import math

import numpy as np
import pytest
import torch

import operands as ref
from test_gpu_cache import cuda, sequences

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def filled(pages, page, heads, dim, seed, garbage=True):
    """A cache of random codes and scales; unused places hold bytes and scales of any kind."""
    r = np.random.default_rng(seed)
    c = ref.Cache(pages, page, heads, dim)
    c.k = r.integers(0, 256, c.k.shape, np.uint8)
    c.v = r.integers(0, 256, c.v.shape, np.uint8)
    c.ks = ref.up5(np.exp(r.normal(0, 0.4, c.ks.shape)) * 0.2)
    c.vs = ref.up5(np.exp(r.normal(0, 0.6, c.vs.shape)) * 0.15)
    return c


def poison(cache, table, length):
    """NaN scales wherever no sequence has a token (a cache never written there)."""
    used = np.zeros((cache.pages, cache.page), bool)
    for b in range(len(length)):
        for pos in range(max(0, int(length[b]))):
            at = cache.place(table, b, pos)
            if at:
                used[at] = True
    for s in (cache.ks, cache.vs):
        s[~used[:, None, :, None].repeat(cache.heads, 1).repeat(cache.G, 3)] = np.nan


def check(gpu, cache, Q, table, length, start, scale=None, window=0, sinks=0, what="", **kw):
    sc = 1.0 / math.sqrt(cache.dim) if scale is None else scale
    want, lse, bound, done = ref.attention(cache, Q, table, length, start, sc, window, sinks)
    out = torch.full(Q.shape, 7.0, dtype=Q.dtype, device="cuda")
    got, l = gpu.gptq_cache_attention(cache.tensors("cuda"), Q, cuda(table), cuda(length), cuda(start), scale, window, sinks, out=out,
                                      want_lse=True, **kw)
    ref.assert_within(got[cuda(done)], want[done], bound[done], what)
    assert (got[cuda(~done)] == 7).all()
    l = l.cpu().numpy()[done]
    assert np.array_equal(np.isneginf(l), np.isneginf(lse[done])), what
    f = np.isfinite(lse[done])
    assert np.all(np.abs(l[f] - lse[done][f]) <= 2e-4 * (1 + np.abs(lse[done][f]))), what
    return got


# lengths, rows (None: one a sequence), page, heads, group
CASES = [([1], None, 16, 1, 1), ([17, 32, 33, 64, 5], None, 16, 2, 4), ([0, 1, 300], None, 32, 1, 16), ([130, 2], [3, 2], 16, 2, 7),
         ([40, 0, 257], [5, 0, 20], 48, 1, 8), ([600], None, 64, 3, 1), ([2000, 31], None, 16, 1, 20), ([96, 130], [96, 70], 16, 1, 3),
         ([700], [260], 64, 1, 4), ([5, 9], [8, 9], 16, 2, 2), ([1100], [1], 16, 2, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(gpu, kind, dim, case):
    lengths, rows, page, heads, group = CASES[case]
    pages = sum(-(-n // page) for n in lengths) + 2
    table, length, start = sequences(lengths, rows if rows else [1] * len(lengths), page, pages, case, single=rows is None)
    cache = filled(pages, page, heads, dim, case)
    poison(cache, table, length)
    total = len(lengths) if rows is None else int(start[-1])
    extra = 0 if rows is None else 3
    Q = torch.randn(total + extra, heads * group, dim, generator=torch.Generator().manual_seed(case)).to(kind).cuda()
    check(gpu, cache, Q, table, length, start, what="causal")
    for window, sinks in ((1, 0), (33, 4), (100, 40)):
        check(gpu, cache, Q, table, length, start, window=window, sinks=sinks, what=f"window {window} sinks {sinks}")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
def test_scales_of_scores(gpu, kind):
    """Scores far apart, all equal, and negated."""
    table, length, start = sequences([500, 300], [40, 1], 16, 60, 1)
    cache = filled(60, 16, 2, 128, 1)
    Q = torch.randn(41, 4, 128, generator=torch.Generator().manual_seed(2)).to(kind).cuda()
    for scale in (0.0, 1.0, -0.3, 1e-3):
        check(gpu, cache, Q, table, length, start, scale=scale, what=f"scale {scale}")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows", [1, 30])
def test_absent_pages(gpu, kind, rows):
    """Pages outside the cache are not seen, wherever they lie; a row with nothing else sees nothing."""
    table, length, start = sequences([200, 40, 100], [rows] * 3, 16, 40, 3)
    cache = filled(40, 16, 2, 64, 3)
    table[0, 0], table[0, 5], table[0, 12] = -1, 40, 2**31 - 1
    table[1, :] = -7
    length[2] = 100000  # past the table
    Q = torch.randn(3 * rows, 4, 64, generator=torch.Generator().manual_seed(3)).to(kind).cuda()
    got = check(gpu, cache, Q, table, length, start, what="absent")
    assert (got[rows:2 * rows] == 0).all()
    check(gpu, cache, Q, table, length, start, window=50, sinks=20, what="absent, window")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_values_not_finite(gpu, rows):
    """A poisoned token reaches the rows that see it and no other; a bad query only its own row."""
    table, length, start = sequences([100], [rows], 16, 8, 4)
    cache = filled(8, 16, 1, 128, 4)
    Q = torch.randn(rows, 2, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    clean = check(gpu, cache, Q, table, length, start)
    bad = Q.clone()
    bad[rows - 1, 1, 3] = float("nan")
    got = gpu.gptq_cache_attention(cache.tensors("cuda"), bad, cuda(table), cuda(length), cuda(start))
    assert torch.isnan(got[rows - 1, 1]).all()
    keep = torch.ones(rows, 2, dtype=torch.bool)
    keep[rows - 1, 1] = False
    assert torch.equal(got[keep.cuda()], clean[keep.cuda()])
    p, o = cache.place(table, 0, 80)
    cache.vs[p, 0, o, 1] = np.nan
    got = gpu.gptq_cache_attention(cache.tensors("cuda"), Q, cuda(table), cuda(length), cuda(start))
    sees = torch.arange(100 - rows, 100) >= 80
    assert torch.isnan(got[sees.cuda()][:, :, 32:64]).all()
    assert torch.equal(got[~sees.cuda()], clean[~sees.cuda()])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 33])
def test_strides_streams_and_in_place(gpu, rows):
    """Slices of a fused projection, heads outside rows, O over Q, another stream: the same bits."""
    table, length, start = sequences([150, 90], [rows, rows], 32, 20, 6)
    cache = filled(20, 32, 2, 64, 6)
    planes, tb, ln, st = cache.tensors("cuda"), cuda(table), cuda(length), cuda(start)
    Q = torch.randn(2 * rows, 6, 64, generator=torch.Generator().manual_seed(7)).to(torch.float16).cuda()
    want = check(gpu, cache, Q, table, length, start)
    fused = torch.randn(2 * rows, 10, 64, device="cuda").half()
    fused[:, 2:8] = Q
    assert torch.equal(gpu.gptq_cache_attention(planes, fused[:, 2:8], tb, ln, st), want)
    outside = Q.transpose(0, 1).contiguous().transpose(0, 1)
    o = torch.empty_like(outside)
    assert torch.equal(gpu.gptq_cache_attention(planes, outside, tb, ln, st, out=o), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = gpu.gptq_cache_attention(planes, Q, tb, ln, st, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, want)
    gpu.gptq_cache_attention(planes, fused[:, 2:8], tb, ln, st, out=fused[:, 2:8])
    assert torch.equal(fused[:, 2:8], want)


@pytest.mark.gpu
def test_pieces_agree_with_shared_prefix(gpu):
    """Two sequences on the same pages give the same rows, and a long one is cut into pieces the same
    way every time."""
    table, length, _ = sequences([3000], [1], 16, 200, 8, single=True)
    cache = filled(200, 16, 1, 128, 8)
    Q = torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    one = check(gpu, cache, Q, table, length, None)
    two = gpu.gptq_cache_attention(cache.tensors("cuda"), Q.repeat(2, 1, 1), cuda(table.repeat(2, 0)), cuda(length.repeat(2)))
    assert torch.equal(two[0], two[1])
    again = gpu.gptq_cache_attention(cache.tensors("cuda"), Q, cuda(table), cuda(length))
    assert torch.equal(one, again)


@pytest.mark.gpu
def test_wild_metadata_stays_inside(gpu):
    cache = filled(3, 16, 1, 64, 9)
    planes = cache.tensors("cuda")
    Q = torch.randn(6, 2, 64, device="cuda")
    table = cuda(np.array([[7, -3], [2**31 - 1, -2**31]], np.int32))
    for length, start in (([2**31 - 1, -2**31], [0, 3, 6]), ([4, 4], [5, 2, 1]), ([20, 20], [-9, 100, 2]), ([1, 1], [7, 8, 9])):
        for window in (0, 5, 2**31 - 1):
            o = gpu.gptq_cache_attention(planes, Q, table, cuda(np.array(length, np.int32)), cuda(np.array(start, np.int32)),
                                         window=window, sinks=2**31 - 1, out=torch.zeros_like(Q))
            assert (o == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [100, 1050, 40000])
@pytest.mark.parametrize("ragged", [False, True])
def test_many_sequences(gpu, ragged, n):
    """Sequences that repeat 50: every repetition has its model's bits.  More of them than a look at their
    starts takes in, and than an axis of a grid."""
    same = 50
    cache = filled(60, 16, 1, 64, 21)
    r = np.random.default_rng(22)
    rows = r.integers(0, 4, same) if ragged else np.ones(same, np.int64)
    rows[7] = 40 if ragged else 1
    table = np.tile(r.permutation(60)[:same].reshape(same, 1).astype(np.int32), (n // same, 1))
    length = np.tile(r.integers(0, 17, same).astype(np.int32), n // same)
    Q = torch.randn(int(rows.sum()), 2, 64, device="cuda", dtype=torch.bfloat16)
    start = np.concatenate([[0], np.cumsum(np.tile(rows, n // same))]).astype(np.int32) if ragged else None
    one = check(gpu, cache, Q, table[:same], length[:same], None if start is None else start[:same + 1])
    got = gpu.gptq_cache_attention(cache.tensors("cuda"), Q.repeat(n // same, 1, 1), cuda(table), cuda(length), cuda(start))
    assert (got.view(n // same, *Q.shape) == one).all()


@pytest.mark.gpu
def test_far_pages(gpu):
    """Pages whose bytes lie past 2^32: the bits of the same pages at the front of a cache."""
    pages, page, heads, dim = 700000, 16, 8, 128
    far = gpu.cache_alloc(pages, page, heads, dim)
    near = gpu.cache_alloc(64, page, heads, dim)
    at = torch.cat([torch.arange(32), torch.arange(pages - 32, pages)]).to(torch.int32)[torch.randperm(64, generator=torch.Generator().manual_seed(1))]
    tables = [at.view(2, 32).cuda(), torch.arange(64, dtype=torch.int32).view(2, 32).cuda()]
    length, start = cuda(np.array([500, 301], np.int32)), cuda(np.array([0, 500, 801], np.int32))
    g = torch.Generator("cuda").manual_seed(2)
    K, V = torch.randn(2, 801, heads, dim, device="cuda", generator=g, dtype=torch.bfloat16).unbind()
    Q = torch.randn(801, 16, dim, device="cuda", generator=g, dtype=torch.bfloat16)
    out = []
    for cache, table in zip((far, near), tables):
        gpu.gptq_cache_write(cache, K, V, table, length, start)
        out.append((*gpu.gptq_cache_read(cache, table, length, start, 801), gpu.gptq_cache_attention(cache, Q, table, length, start),
                    gpu.gptq_cache_attention(cache, Q[:2], table, length)))
    assert cache[0].any() and far[0][-32:].any()
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_refusals(gpu):
    planes = gpu.cache_alloc(2, 16, 2, 64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    length = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, 64, device="cuda")
    for kw in (dict(Q=q[..., :32]), dict(Q=q.double()), dict(Q=q[0]), dict(Q=q.cpu()), dict(out=q.half()), dict(table=table.long()),
               dict(Q=q.repeat(2, 1, 1)), dict(workspace=torch.empty(3, device="cuda"), table=table.repeat(1, 4000)), dict(window=1 << 32), dict(sinks=1 << 31),
               dict(window=-(1 << 32))):
        args = dict(cache=planes, Q=q, table=table, length=length)
        args.update(kw)
        with pytest.raises(ValueError):
            gpu.gptq_cache_attention(**args)
    for kw in (dict(Q=q[:, :3]), dict(window=-1), dict(sinks=-1), dict(scale=float("nan"))):
        args = dict(cache=planes, Q=q, table=table, length=length)
        args.update(kw)
        with pytest.raises(gpu.GptqError):
            gpu.gptq_cache_attention(**args)
