"""Rotary positions against their definition in 64 bits: types, layouts, odd sizes, far positions, in place, slices of
one projection, heads outside rows, the backward pass, graphs."""
import pytest
import torch

import layer
import operands as ref

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(rows, heads, dim, kind, seed, far=4096):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads, dim, generator=g).to(kind).cuda()
    return x, torch.randint(0, far, (rows,), generator=g, dtype=torch.int32).cuda()


def check(got, x, p, f, layout, factor, backward, what):
    want, bound = layer.rotary(x, p, f, layout, factor, backward)
    ref.assert_within(got, want, bound, what)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rows,hq,hk,dim,part", [(1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (48, 7, 1, 80, 80), (5, 3, 2, 81, 80), (33, 4, 4, 96, 26),
                                                 (700, 5, 1, 64, 16), (3, 2, 1, 256, 255 - 1), (2, 1, 1, 2048, 2048), (2, 3, 1, 33, 2),
                                                 (9000, 2, 1, 64, 64), (5000, 1, 2, 20, 18)])
def test_sizes(gpu, kind, layout, rows, hq, hk, dim, part):
    (q, p), (k, _) = make(rows, hq, dim, kind, rows + dim), make(rows, hk, dim, kind, rows)
    f, factor = gpu.rotary_frequencies(part, scaling="ramp" if part > 2 else "none", stretch=4.0)
    for backward in (False, True):
        a, b = gpu.gptq_rotary(q, p, f, K=k, layout=layout, factor=factor, backward=backward)
        check(a, q, p, f, layout, factor, backward, "Q")
        check(b, k, p, f, layout, factor, backward, "K")
    assert torch.equal(gpu.gptq_rotary(q, p, f, layout=layout, factor=factor), gpu.gptq_rotary(q, p, f, K=k, layout=layout, factor=factor)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,part,shift", [(64, 64, 0), (64, 32, 0), (64, 32, 1), (24, 10, 0)])
def test_slices_in_place(gpu, kind, layout, dim, part, shift):
    """Queries and keys of one projection, turned where they lie; its values, and what is between, stay."""
    rows, hq, hk = 37, 4, 2
    buf, p = make(rows, 1, (hq + 2 * hk) * dim + 8, kind, 3)
    x = buf.view(rows, -1)
    before = x.clone()
    q, k = (x[:, shift + o:shift + o + h * dim].unflatten(1, (h, dim)) for o, h in ((0, hq), (hq * dim, hk)))
    f, factor = gpu.rotary_frequencies(part)
    cq, ck = q.clone(), k.clone()
    out = gpu.gptq_rotary(q, p, f, K=k, layout=layout, factor=factor, out=(q, k))
    assert out[0] is q and out[1] is k
    check(q, cq, p, f, layout, factor, False, "Q")
    check(k, ck, p, f, layout, factor, False, "K")
    end = shift + (hq + hk) * dim
    assert torch.equal(x[:, :shift], before[:, :shift]) and torch.equal(x[:, end:], before[:, end:])
    if part < dim:
        assert torch.equal(q[..., part:], cq[..., part:])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_heads_outside_rows(gpu, layout):
    x, p = make(3, 40, 64, torch.bfloat16, 5)
    q = x.transpose(0, 1)  # [40 rows, 3 heads, 64]
    p = torch.arange(40, dtype=torch.int32, device="cuda")
    f, _ = gpu.rotary_frequencies(64)
    check(gpu.gptq_rotary(q, p, f, layout=layout), q, p, f, layout, 1.0, False, "heads first")
    keep = q.clone()
    gpu.gptq_rotary(q, p, f, layout=layout, out=q)
    check(q, keep, p, f, layout, 1.0, False, "in place")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(gpu, layout):
    """Angles of up to 2^31 turns, negative positions, and a frequency of nothing."""
    x, _ = make(9, 2, 64, torch.float32, 7)
    p = torch.tensor([0, 1, -1, 131071, 1 << 20, (1 << 31) - 1, -(1 << 31), 999999937, -5], dtype=torch.int32, device="cuda")
    f, _ = gpu.rotary_frequencies(64)
    f[3] = 0.0
    y = gpu.gptq_rotary(x, p, f, layout=layout)
    want, bound = layer.rotary(x, p, f, layout, 1.0, False)
    # The definition's own angles are f64: 2^-53 of up to 2^31.
    ref.assert_within(y, want, bound + 2.0 ** -20 * (p.double().cpu().abs() > 1 << 24)[:, None, None] * want.abs().amax(), "far")
    assert torch.equal(y[0], x[0])


@pytest.mark.gpu
def test_infinities_and_nothing(gpu):
    x, p = make(4, 2, 64, torch.float32, 9)
    f, _ = gpu.rotary_frequencies(32)
    clean = gpu.gptq_rotary(x, p, f)
    x[1, 0, 3] = float("nan")
    x[2, 1, 60] = float("inf")
    y = gpu.gptq_rotary(x, p, f)
    same = ~torch.isnan(y)
    same[2, 1, 60] = False
    assert torch.equal(y[same], clean[same]) and torch.isnan(y).nonzero().tolist() == [[1, 0, 3], [1, 0, 19]]
    assert y[2, 1, 60] == float("inf")
    assert gpu.gptq_rotary(x[:0], p[:0], f).shape == (0, 2, 64)
    with pytest.raises(gpu.GptqError):
        gpu.gptq_rotary(x, p, f, out=x[:, :1].expand(4, 2, 64))
    with pytest.raises(gpu.GptqError):
        gpu.gptq_rotary(x, p, torch.zeros(40, dtype=torch.float64, device="cuda"))


@pytest.mark.gpu
def test_captured(gpu):
    x, p = make(48, 5, 128, torch.bfloat16, 11)
    f, _ = gpu.rotary_frequencies(128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = gpu.gptq_rotary(x, p, f, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, gpu.gptq_rotary(x, p, f))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gpu.gptq_rotary(x, p, f)
    for i in range(5):
        p.add_(1)
        graph.replay()
        got = y.clone()
        assert torch.equal(got, gpu.gptq_rotary(x, p, f)), i
