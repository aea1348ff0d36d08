"""The 4-bit cache written and read back (gptq_cache_write, gptq_cache_read) against the stated
bytes and values: every type and size, values at the borders of codes, odd lengths, absent pages,
rows behind the last sequence, and what must stay as it was."""
import numpy as np
import pytest
import torch

import operands as ref

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def sequences(lengths, rows, page, pages, seed, single=False):
    """Table, lengths and starts of sequences on pages without order."""
    r = np.random.default_rng(seed)
    width = max(1, max(-(-n // page) for n in lengths))
    table = np.full((len(lengths), width), -1, np.int32)
    order = list(r.permutation(pages))
    for b, n in enumerate(lengths):
        for i in range(-(-n // page)):
            table[b, i] = order.pop()
    start = None if single else np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return table, np.array(lengths, np.int32), start


def cuda(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bits(x):
    return x.view({2: torch.int16, 4: torch.int32, 1: torch.uint8}[x.element_size()])


CASES = [  # lengths, rows, page, heads
    ([1], [1], 16, 1), ([5, 0, 33], [5, 0, 33], 16, 3), ([40, 16, 1, 300], [7, 16, 1, 129], 32, 2),
    ([70] * 70, [1] * 70, 16, 2), ([2, 64], [2, 1], 64, 5), ([130], [100], 48, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_write_and_read(gpu, kind, dim, case):
    lengths, rows, page, heads = CASES[case]
    pages = sum(-(-n // page) for n in lengths) + 2
    table, length, start = sequences(lengths, rows, page, pages, case)
    total = int(start[-1])
    g = torch.Generator().manual_seed(case * 31 + dim)
    x = torch.randn(total + 2, 2, heads, dim, generator=g) * torch.exp(torch.randn(total + 2, 2, heads, 1, generator=g) * 3)
    x = x.to(kind).cuda()
    K, V = x[:, 0], x[:, 1]
    want = ref.Cache(pages, page, heads, dim, fill=0xA5)
    planes = want.tensors("cuda")
    want.write(table, length, start, K[:total].double().cpu().numpy(), V[:total].double().cpu().numpy())
    # Two rows behind the last sequence are in the call.
    gpu.gptq_cache_write(planes, K, V, cuda(table), cuda(length), cuda(start))
    for got, exp, name in zip(planes, want.tensors("cuda"), ("k", "v", "k_scale", "v_scale")):
        assert torch.equal(bits(got), bits(exp)), name
    out = torch.full((2, total + 2, heads, dim), 7.0, dtype=kind, device="cuda")
    k, v = gpu.gptq_cache_read(planes, cuda(table), cuda(length), cuda(start), rows=total + 2, out=(out[0], out[1]))
    assert (out[:, total:] == 7).all()
    for got, src in ((k, K), (v, V)):
        c, s = ref.quantize(src[:total].double().cpu().numpy())
        val = torch.from_numpy(c * np.repeat(s, 32, -1))
        if kind is torch.float16:
            val = val.clamp(-65504, 65504)
        assert torch.equal(got[:total].cpu(), val.to(kind)), "values"
    # Read again in bf16, which holds every code exactly.
    k16, _ = gpu.gptq_cache_read(planes, cuda(table), cuda(length), cuda(start), rows=total, dtype=torch.bfloat16)
    c, s = ref.quantize(K[:total].double().cpu().numpy())
    assert torch.equal(k16.double().cpu(), torch.from_numpy(c * np.repeat(s, 32, -1)))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
def test_borders(gpu, kind):
    """Groups whose values lie on and next to the borders between codes, and of every magnitude."""
    rows = []
    r = np.random.default_rng(3)
    for e in list(range(-20, 15)) + ([] if kind is torch.float16 else [-140, -133, -126, -100, 90, 120, 126]):
        for top in (7.0, 7.25, 6.9, 1.0, 13.5):
            v = np.concatenate([[top], np.arange(-6.5, 7.0) * up(top), r.uniform(-top, top, 17)])[:32]
            rows.append(v * 2.0 ** e)
    x = torch.tensor(np.array(rows), dtype=torch.float64)
    x = x.clamp(-torch.finfo(kind).max, torch.finfo(kind).max).to(kind)
    # Neighbours of the borders too.
    x = torch.cat([x, bits_step(x, 1), bits_step(x, -1)]).repeat_interleave(2, 0).reshape(-1, 1, 64)
    n = x.shape[0]
    planes = gpu.cache_alloc(-(-n // 16), 16, 1, 64)
    table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None]
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    xd = x.cuda()
    gpu.gptq_cache_write(planes, xd, xd, table, length, start)
    c, s = ref.quantize(x.double().numpy())
    k, v = gpu.gptq_cache_read(planes, table, length, start, rows=n, dtype=torch.float32)
    val = torch.from_numpy(c * np.repeat(s, 32, -1)).float()
    for got in (k.cpu(), v.cpu()):  # the largest magnitudes pass 2^127: NaN on both sides
        assert torch.equal(torch.isnan(got), torch.isnan(val))
        assert torch.equal(got.nan_to_num(9.0), val.nan_to_num(9.0))


def up(top):
    return float(ref.up5(np.array(top / 7.0)))


def bits_step(x, d):
    """The type's neighbour of each value that is not zero and not its largest."""
    b = bits(x.contiguous()).clone()
    top = bits(torch.tensor([torch.finfo(x.dtype).max], dtype=x.dtype))[0]
    mag = b & top.new_tensor(torch.iinfo(b.dtype).max)
    ok = (mag > 1) & (mag < top - 1)
    return torch.where(ok, b + d, b).view(x.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
def test_not_finite_and_zero(gpu, kind):
    """A group with a value that is not finite reads back as NaN, alone; zeros as zeros."""
    x = torch.randn(16, 2, 128, generator=torch.Generator().manual_seed(1)).to(kind)
    x[0, 0, 5] = float("nan")
    x[1, 1, 33] = float("inf")
    x[2, 0, 127] = float("-inf")
    x[3, 1, 64:96] = 0.0
    x[4, 0] = -0.0
    if kind is not torch.float16:
        x[5, 0, 0] = 2.0 ** 127
        x[6, 0, 0] = 2.0 ** 126
        x[7, 0, 32:64] = 1e-40
    planes = gpu.cache_alloc(1, 16, 2, 128)
    ar = dict(table=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), length=torch.tensor([16], dtype=torch.int32, device="cuda"),
              start=torch.tensor([0, 16], dtype=torch.int32, device="cuda"))
    xd = x.cuda()
    gpu.gptq_cache_write(planes, xd, xd, **ar)
    c, s = ref.quantize(x.double().numpy())
    val = torch.from_numpy(c * np.repeat(s, 32, -1)).to(kind)
    for got in gpu.gptq_cache_read(planes, rows=16, dtype=kind, **ar):
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(val)) and torch.equal(got.nan_to_num(9.0), val.nan_to_num(9.0))
    assert torch.isnan(val[0, 0, :32]).all() and not torch.isnan(val[0, 0, 32:]).any()


@pytest.mark.gpu
def test_absent_pages_and_single_rows(gpu):
    """Rows without a place are dropped and read as zeros; nothing else changes."""
    page, heads, dim = 16, 2, 64
    want = ref.Cache(4, page, heads, dim, fill=0x11)
    planes = want.tensors("cuda")
    table = np.array([[0, 9], [2, 1], [-1, 3], [3, 2]], np.int32)
    length = np.array([20, 33, 5, 0], np.int32)  # on page 9; past the table; on page -1; before the sequence
    x = torch.randn(4, 2, heads, dim).cuda()
    before = [t.clone() for t in planes]
    gpu.gptq_cache_write(planes, x[:, 0], x[:, 1], cuda(table), cuda(length))
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(planes, before))
    k, v = gpu.gptq_cache_read(planes, cuda(table), cuda(length), dtype=torch.float32)
    assert (k == 0).all() and (v == 0).all()
    length = np.array([16, 32, 20, 1], np.int32)
    want.write(table, length, None, x[:, 0].double().cpu().numpy(), x[:, 1].double().cpu().numpy())
    gpu.gptq_cache_write(planes, x[:, 0], x[:, 1], cuda(table), cuda(length))
    for got, exp in zip(planes, want.tensors("cuda")):
        assert torch.equal(bits(got), bits(exp))


@pytest.mark.gpu
def test_wild_metadata_stays_inside(gpu):
    """Lengths and starts of any value: what has no place is skipped."""
    want = ref.Cache(3, 16, 1, 64, fill=0x77)
    planes = want.tensors("cuda")
    before = [t.clone() for t in planes]
    x = torch.randn(6, 2, 1, 64).cuda()
    table = cuda(np.array([[7, -3], [2**31 - 1, -2**31]], np.int32))
    for length, start in (([2**31 - 1, -2**31], [0, 3, 6]), ([4, 4], [5, 2, 1]), ([20, 20], [-9, 100, 2]), ([1, 1], [7, 8, 9])):
        ln, st = cuda(np.array(length, np.int32)), cuda(np.array(start, np.int32))
        gpu.gptq_cache_write(planes, x[:, 0], x[:, 1], table, ln, st)
        out = torch.full((2, 6, 1, 64), 5.0, device="cuda")
        gpu.gptq_cache_read(planes, table, ln, st, rows=6, out=(out[0], out[1]))
        assert ((out == 0) | (out == 5)).all()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(planes, before))


@pytest.mark.gpu
def test_refusals(gpu):
    planes = gpu.cache_alloc(2, 16, 2, 64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    length = torch.ones(1, dtype=torch.int32, device="cuda")
    x = torch.randn(1, 2, 64, device="cuda")
    for kw in (dict(K=x[:, :1]), dict(V=x.half()), dict(K=x.double(), V=x.double()), dict(table=table.long()), dict(length=length[:0]),
               dict(table=table[0]), dict(start=torch.zeros(1, dtype=torch.int32, device="cuda")), dict(K=x.cpu()),
               dict(cache=(planes.k, planes.v[:1], planes.k_scale, planes.v_scale)),
               dict(cache=(planes.k, planes.v, planes.k_scale.half(), planes.v_scale)),
               dict(K=torch.randn(3, 2, 64, device="cuda"), V=torch.randn(3, 2, 64, device="cuda"))):
        args = dict(cache=planes, K=x, V=x, table=table, length=length)
        args.update(kw)
        with pytest.raises(ValueError):
            gpu.gptq_cache_write(**args)
    with pytest.raises(ValueError):
        gpu.gptq_cache_read(planes, table, length, rows=2)
