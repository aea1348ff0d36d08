"""Precision of the layer's further operators where sums, ranges and angles are hard: errors over a whole result against 64
bits, held to what the stated roundings give."""
import numpy as np
import pytest
import torch

import layer
import operands as ref
from test_gpu_gated import make


def off(got, want):
    """The error's norm over the result's."""
    return float((got.double().cpu() - want).norm() / want.norm())


def rounding(want, kind):
    """What one rounding to the type puts a result off by."""
    return float((want.to(kind).double() - want).norm() / want.norm())


def balanced(rows, n, g):
    """q4tp codes 1 .. 15, whose levels cancel on average."""
    nib = torch.randint(1, 16, (2, rows, n // 2), generator=g, dtype=torch.uint8)
    return (nib[0] | nib[1] << 4).cuda(), torch.exp2(torch.randn(rows, n // 32, generator=g) * 0.5 - 6.0).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,rows,n", [(1536, 17408, 2048), (3060, 33000, 1024), (16, 33000, 4096)])
def test_gradients_of_one_sign(gpu, kind, t, rows, n):
    """Gradients that do not cancel, over many rows that one wave sums: what the codes' offset adds to f32 sums on
    the way grows with the rows, the result with their root.  dY times a scale is rounded to 2^-16, far below the
    result's own rounding."""
    g = torch.Generator().manual_seed(rows)
    dY = torch.randn(t, rows, generator=g).abs().to(kind).cuda()
    codes, scale = balanced(rows, n, g)
    got = gpu.gptq_linear_backward(dY, codes, scale, exact=True)
    pick = torch.arange(0, t, max(1, t // 48))
    want = dY[pick.cuda()].double().cpu() @ ref.weight_values(codes, scale, "q4tp")
    assert off(got[pick.cuda()], want) < 1.1 * rounding(want, kind)


# f32 sums: a step's 32 products are added up in f32, in up to four parts of each of three terms, cut rather than rounded
# at worst: sqrt(12) times 2^-23 / sqrt(3) of a step's sum, 2^-23 2 over all steps; the steps' sums join those before them
# one by one, a random walk of at most 2^-24 / sqrt(3) sqrt(steps / 2), 64 steps here: 2^-24 3.3.  Together below
# 2^-24 5.2; the terms' last roundings and the result's are 2^-24 each at most.
F32 = 2.0 ** -21


@pytest.mark.gpu
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", [(37, 2048, 2048), (16, 513, 4096), (333, 1024, 1024), (128, 70, 8192)])
def test_f32_gradients_as_exact_as_f32_sums(gpu, codec, t, rows, n):
    _, dY, gate, _, _ = make(t, rows, n, torch.float32, codec, 5)
    assert off(gpu.gptq_linear_backward(dY, *gate, codec), layer.linear_backward(dY, *gate, codec)[0]) < F32


@pytest.mark.gpu
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("t,rows,n", [(2, 774, 416), (16, 513, 2080), (200, 130, 992), (300, 515, 1504), (64, 4100, 2048)])
def test_f32_block_as_exact_as_f32_sums(gpu, codec, t, rows, n):
    """The sums of both matrices at F32, their product sqrt(2) times that; the gradient's own sums once more."""
    X, dY, gate, up, _ = make(t, rows, n, torch.float32, codec, 6)
    y = gpu.gptq_gated(X, gate, up, codec, "none")
    assert off(y, layer.gated(X, gate, up, codec, "none", (None, None))[0]) < 1.42 * F32
    dx = gpu.gptq_gated_backward(dY, X, gate, up, codec, "none")
    assert off(dx, layer.gated_backward(dY, X, gate, up, codec, "none", (None, None))[0]) < 1.74 * F32


@pytest.mark.gpu
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("t,rows,n", [(1210, 2101, 2080), (600, 4100, 2144), (3300, 1030, 1568)])
def test_f16_prompts(gpu, codec, act, t, rows, n):
    """On decoded weights an f16 result of two products is off by its own rounding, as one of f32 sums is; the gradient
    of X by one more like it, that of the last product's weights to 11 bits."""
    X, dY, gate, up, _ = make(t, rows, n, torch.float16, codec, 7)
    X, dY = (X * 0.125).half(), (dY * 16).half()
    y, dx = gpu.gptq_gated(X, gate, up, codec, act), gpu.gptq_gated_backward(dY, X, gate, up, codec, act)
    want = layer.gated(X, gate, up, codec, act, (None, None))[0]
    assert off(y, want) < 1.1 * rounding(want, torch.float16)
    want = layer.gated_backward(dY, X, gate, up, codec, act, (None, None))[0]
    assert off(dx, want) < 1.5 * rounding(want, torch.float16)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act,low", [("silu", -1e9), ("gelu", -1e30), ("gelu_tanh", -3e38), ("relu", -1e30), ("relu", float("-inf"))])
def test_gates_shut_by_their_bias(gpu, kind, act, low):
    """A gate that a large negative bias shuts takes no part, and leaves the others their precision: results are those of
    the block whose gradients there are zeros, its bounds too."""
    t, rows, n = 1210, 2101, 2080
    X, dY, gate, up, bias = make(t, rows, n, kind, "q4tp", 8)
    shut = torch.arange(rows, device="cuda") % 5 == 2
    masked = torch.where(shut, torch.tensor(low, device="cuda"), bias[0])
    y = gpu.gptq_gated(X, gate, up, "q4tp", act, masked, bias[1])
    assert (y[:, shut] == 0).all()
    dx = gpu.gptq_gated_backward(dY, X, gate, up, "q4tp", act, masked, bias[1])
    want, bound = layer.gated_backward(torch.where(shut, 0.0, dY).to(kind), X, gate, up, "q4tp", act, bias)
    ref.assert_within(dx, want, bound, act)
    assert off(dx, want) < 2.0 * rounding(want, kind)


def turn_part(position, freq):
    """position freq / 2 pi less its nearest whole number, in rationals; pi from Machin's formula, 70 digits."""
    from fractions import Fraction
    one = 10 ** 70

    def arctan_of(k):
        s, x, n = 0, one // k, 0
        while x:
            s += (x // (2 * n + 1)) * (-1) ** n
            x //= k * k
            n += 1
        return s

    pi = Fraction(4 * (4 * arctan_of(5) - arctan_of(239)), one)
    v = Fraction(int(position)) * Fraction(float(freq)) / (2 * pi)
    return float(v - round(v))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_cosines_of_far_positions(gpu, layout):
    """Pairs (1, 0) in f32 become cosine and sine: off by the angle's rounding to f32 (2^-25 of a half turn: 2^-25 pi) and
    two units of the last place of the functions (2^-23), wherever the position lies."""
    p = [0, 1, 7, 4095, 131071, 1 << 20, (1 << 26) + 1, 999999937, (1 << 30) - 35, (1 << 31) - 1, -1, -123456789, -(1 << 31)]
    f, _ = gpu.rotary_frequencies(128)
    f = torch.cat([f, torch.tensor([3.0, 0.999], dtype=torch.float64, device="cuda")])
    half = f.shape[0]
    x = torch.zeros(len(p), 1, 2 * half, device="cuda")
    i0 = torch.arange(half) if layout == "half" else 2 * torch.arange(half)
    i1 = i0 + (half if layout == "half" else 1)
    x[..., i0] = 1.0
    y = gpu.gptq_rotary(x, torch.tensor(p, dtype=torch.int32, device="cuda"), f, layout=layout).double().cpu()
    turns = 2 * np.pi * np.array([[turn_part(a, b) for b in f.cpu()] for a in p])
    worst = max(np.abs(y[:, 0, i0].numpy() - np.cos(turns)).max(), np.abs(y[:, 0, i1].numpy() - np.sin(turns)).max())
    assert worst <= 2.0 ** -25 * np.pi + 2.0 ** -23, worst


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_of_many_rows(gpu, kind, dim):
    """32768 query rows over tokens that all weigh about the same, so that neither the scale's rounding nor one weight's
    shows: each token's sum is off by its own rounding and that of joining eight parts (up to 2^-24 each,
    at the sum's size the last three)."""
    R, group, past, page = 4096, 8, 64, 64
    L = R + past
    pages = L // page
    r = np.random.RandomState(dim)
    c = ref.Cache(pages, page, 1, dim)
    c.k[:] = r.randint(1, 16, c.k.shape) | r.randint(1, 16, c.k.shape) << 4
    c.ks[:] = c.vs[:] = 2.0 ** -6
    table = r.permutation(pages).astype(np.int32)[None]
    Q = (torch.randn(R, group, dim, generator=torch.Generator().manual_seed(1)) * 0.02).to(kind).cuda()
    K = torch.from_numpy(c.values(table, 0, L)[0][:, 0]).cuda()
    seen = torch.arange(L, device="cuda")[None, None] <= past + torch.arange(R, device="cuda")[:, None, None]
    want, lse = torch.zeros(L, dtype=torch.float64, device="cuda"), torch.empty(R, group, device="cuda")
    for r0 in range(0, R, 256):
        s = (Q[r0:r0 + 256].double().flatten(0, 1) @ K.t()).view(-1, group, L) * dim ** -0.5
        s = s.masked_fill(~seen[r0:r0 + 256], float("-inf"))
        lse[r0:r0 + 256] = torch.logsumexp(s, -1)
        want += torch.exp(s - lse[r0:r0 + 256].double()[..., None]).sum((0, 1))
    args = [torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in (table, [L], [0, R])]
    out = gpu.gptq_cache_score(c.tensors("cuda"), Q, lse, torch.zeros(pages, 1, page, device="cuda"), *args)
    got = out[args[0][0].long()].flatten()
    assert off(got, want.cpu()) < 1.5 * 2.0 ** -24


@pytest.mark.gpu
def test_scores_past_a_grid_of_pieces(gpu):
    """A table so long, beside so many heads and sequences, that a workgroup takes a second piece of its sequence: tokens on
    both sides of the 131200 that the first pieces reach, most of the table's pages absent."""
    heads, page, dim, R, L = 64, 16, 64, 3, 131200 + 777
    c = ref.Cache(140, page, heads, dim)
    r = np.random.RandomState(4)
    c.k[:] = r.randint(1, 16, c.k.shape) | r.randint(1, 16, c.k.shape) << 4
    c.ks[:] = np.ldexp(r.randint(16, 32, c.ks.shape), -7)
    width = -(-L // page)
    table = np.full((16, width), -1, np.int32)
    there = list(range(3)) + list(range(8190, width))
    table[0, there] = r.permutation(120)[:len(there)]
    table[1:, 0] = 120 + np.arange(15)
    length, start = np.full(16, 9), np.arange(17) + 2
    length[0], start[0] = L, 0
    start[1:] = R + np.arange(16)
    g = torch.Generator().manual_seed(2)
    Q = torch.randn(R + 15, heads, dim, generator=g).cuda()
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    planes, args = c.tensors("cuda"), (i32(table), i32(length), i32(start))
    _, lse = gpu.gptq_cache_attention(planes, Q, *args, want_lse=True)
    old = torch.rand(140, heads, page, generator=g).cuda()
    out = gpu.gptq_cache_score(planes, Q, lse, old, *args, out=torch.full_like(old, -3.0))
    K = torch.from_numpy(c.values(table[:, there][:1], 0, len(there) * page)[0])  # [tokens, heads, dim]
    tok = torch.tensor([p * page + o for p in there for o in range(page)])
    s = torch.einsum("rhd,thd->rht", Q[:R].double().cpu(), K) * dim ** -0.5
    l = lse[:R].double().cpu()[..., None]
    seen = (tok[None] <= L - R + torch.arange(R)[:, None])[:, None]
    w = torch.where(seen, torch.exp(s - l), 0.0)
    spread = torch.einsum("rhd,thd->rht", Q[:R].double().abs().cpu(), K.abs()) * dim ** -0.5
    err = (w * (2 * (40 * 2.0 ** -23 * spread + 2.0 ** -21 * (s.abs() + l.abs() + 2)) + 2.0 ** -20)).sum(0).t()
    at, place = i32(table[0, there]).long().repeat_interleave(page).cpu(), tok % page
    was = torch.where(tok < L - R, 1.0, 0.0)[:, None] * old.double().cpu()[at, :, place]
    want = was + w.sum(0).t()
    got = out.cpu()[at, :, place]
    live = tok < L
    ref.assert_within(got[live], want[live], (err + 2.0 ** -22 * want)[live], "score")
    assert (got[~live] == -3).all()
    for b in range(1, 16):
        assert (out[table[b, 0], :, :8] > old[table[b, 0], :, :8]).all() and (out[table[b, 0], :, 9:] == -3).all()
