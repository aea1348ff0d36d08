"""The layer's further operators without a GPU: their launches by the dry run, their refusals, and arguments that
share memory."""
import random

import pytest
import torch

import post_weight_quantization_amd as pwq
from test_operands_alias import bytes_of
from test_operands_host import addr, batch, cache, lib, raw  # noqa: F401

SIZES = [(1, 1, 32), (1, 4096, 4096), (3, 33, 96), (17, 200, 4128), (64, 48, 160), (333, 2048, 8192), (4096, 5120, 17408),
         (300, 4099, 2080), (40000, 333, 1120), (20000, 5, 64)]


def back(lib, **kw):
    d = dict(D=addr(0), ldd=None, dtype=1, t=5, codec=0, codes=addr(1), scale=addr(2), rows=33, n=96, X=addr(3), ldx=None,
             ws=addr(4), wsb=None)
    d.update(kw)
    d["ldd"] = d["rows"] if d["ldd"] is None else d["ldd"]
    d["ldx"] = d["n"] if d["ldx"] is None else d["ldx"]
    if d["wsb"] is None:
        d["wsb"] = lib.gptq_linear_backward_workspace_size(d["dtype"], d["t"], d["rows"], d["n"])
    with pwq.check_mode():
        return lib.gptq_linear_backward(d["D"], d["ldd"], d["dtype"], d["t"], d["codec"], d["codes"], d["scale"], d["rows"], d["n"],
                                        d["X"], d["ldx"], d["ws"], d["wsb"], None)


def gated(lib, backward=False, **kw):
    d = dict(X=addr(0), ldx=None, dtype=1, t=5, codec=0, g=addr(1), gs=addr(2), gb=addr(3), u=addr(4), us=addr(5), ub=addr(6),
             rows=33, n=96, act=2, Y=addr(7), ldy=None, D=addr(8), ldd=None, ws=addr(9), wsb=None)
    d.update(kw)
    d["ldx"] = d["n"] if d["ldx"] is None else d["ldx"]
    d["ldd"] = d["rows"] if d["ldd"] is None else d["ldd"]
    d["ldy"] = (d["n"] if backward else d["rows"]) if d["ldy"] is None else d["ldy"]
    size = lib.gptq_gated_backward_workspace_size if backward else lib.gptq_gated_workspace_size
    if d["wsb"] is None:
        d["wsb"] = size(d["dtype"], d["t"], d["rows"], d["n"])
    w = [pwq._WEIGHTS(*(v or 0 for v in x)) if x[0] != "none" else None
         for x in ((d["g"], d["gs"], d["gb"]), (d["u"], d["us"], d["ub"]))]
    args = (d["X"], d["ldx"], d["dtype"], d["t"], d["codec"], *w, d["rows"], d["n"], d["act"], d["Y"], d["ldy"], d["ws"], d["wsb"], None)
    with pwq.check_mode():
        return lib.gptq_gated_backward(d["D"], d["ldd"], *args) if backward else lib.gptq_gated(*args)


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("codec", [0, 1])
@pytest.mark.parametrize("t,rows,n", SIZES)
def test_schedules(lib, dtype, codec, t, rows, n):  # noqa: F811
    sizes = dict(dtype=dtype, codec=codec, t=t, rows=rows, n=n)
    assert back(lib, **sizes) == pwq.GPTQ_OK, pwq.check_message()
    assert back(lib, **sizes, ldd=rows + 8, ldx=n + 3) == pwq.GPTQ_OK, pwq.check_message()
    for backward in (False, True):
        assert gated(lib, backward, **sizes) == pwq.GPTQ_OK, pwq.check_message()
        assert gated(lib, backward, **sizes, gb=None, ub=None, ldx=n + 64, ldy=max(rows, n) + 5, ldd=rows + 1) == pwq.GPTQ_OK, pwq.check_message()


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(dtype=-1), dict(t=-1), dict(t=(1 << 24) + 1), dict(codec=2), dict(codec=-1),
                                 dict(D=None), dict(codes=None), dict(scale=None), dict(X=None), dict(rows=0), dict(rows=(1 << 23) + 1),
                                 dict(n=0), dict(n=40), dict(n=(1 << 20) + 32), dict(t=1 << 20, rows=1 << 19), dict(t=1 << 20, n=1 << 19),
                                 dict(ldd=32), dict(ldx=95), dict(D=addr(0) + 1), dict(X=addr(3) + 1), dict(codes=addr(1) + 8),
                                 dict(scale=addr(2) + 2), dict(ws=addr(4) + 64)])
def test_backward_refuses(lib, bad):  # noqa: F811
    assert back(lib, **bad, **({} if "wsb" in bad else dict(wsb=1 << 39))) == pwq.GPTQ_EINVAL


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", [dict(dtype=3), dict(dtype=16 | 3), dict(dtype=32 | 1), dict(t=-1), dict(t=(1 << 24) + 1), dict(codec=2), dict(act=5), dict(act=-1),
                                 dict(X=None), dict(Y=None), dict(g=None), dict(us=None), dict(g="none"), dict(u="none"), dict(rows=0),
                                 dict(rows=(1 << 22) + 1), dict(n=33), dict(n=0), dict(t=1 << 20, rows=1 << 19), dict(t=1 << 20, n=1 << 19),
                                 dict(ldx=95), dict(ldx=100), dict(ldx=(1 << 22) + 8), dict(ldy=32), dict(X=addr(0) + 8), dict(g=addr(1) + 8),
                                 dict(u=addr(4) + 4), dict(gs=addr(2) + 1), dict(ub=addr(6) + 2), dict(Y=addr(7) + 1)])
def test_gated_refuses(lib, backward, bad):  # noqa: F811
    assert gated(lib, backward, **bad, wsb=1 << 39) == pwq.GPTQ_EINVAL


def test_gated_backward_refuses(lib):  # noqa: F811
    for bad in (dict(D=None), dict(ldd=32), dict(D=addr(8) + 1)):
        assert gated(lib, True, **bad, wsb=1 << 39) == pwq.GPTQ_EINVAL


def test_workspaces(lib):  # noqa: F811
    sizes = (lib.gptq_linear_backward_workspace_size, lib.gptq_gated_workspace_size, lib.gptq_gated_backward_workspace_size)
    for size in sizes:
        for args in ((3, 5, 5, 64), (1, -1, 5, 64), (1, 0, 5, 64), (1, 5, 0, 64), (1, 5, 5, 65)):
            assert size(*args) == 0
    calls = (back, lambda lib, **k: gated(lib, False, **k), lambda lib, **k: gated(lib, True, **k))
    for size, call, name in zip(sizes, calls, (4, 9, 9)):
        for t, rows, n, dtype in ((4096, 5120, 17408, 1), (37, 2048, 8192, 0), (20, 4096, 9000 // 32 * 32, 2)):
            need = size(dtype, t, rows, n)
            if need:
                s = dict(t=t, rows=rows, n=n, dtype=dtype)
                assert call(lib, **s, wsb=need - 1) == pwq.GPTQ_EWORKSPACE
                assert call(lib, **s, ws=None, wsb=0) == pwq.GPTQ_EWORKSPACE
                assert call(lib, **s, ws=addr(name) + 16, wsb=need) == pwq.GPTQ_EINVAL
    assert pwq.linear_backward_workspace_size(4096, 5120, 17408) == sizes[0](1, 4096, 5120, 17408)
    assert pwq.gated_workspace_size(4096, 5120, 17408, torch.float16) == sizes[1](2, 4096, 5120, 17408)
    assert pwq.gated_workspace_size(4096, 5120, 17408, backward=True) == sizes[2](1, 4096, 5120, 17408)


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("t,rows,n", [(4096, 5120, 17408), (20000, 333, 1120)])
def test_exact_weights(lib, dtype, t, rows, n):  # noqa: F811
    """No weights decoded in the workspace."""
    sizes = dict(dtype=16 | dtype, t=t, rows=rows, n=n)
    assert back(lib, **sizes) == pwq.GPTQ_OK, pwq.check_message()
    for backward in (False, True):
        assert gated(lib, backward, **sizes) == pwq.GPTQ_OK, pwq.check_message()
    kind = (torch.float32, torch.bfloat16, torch.float16)[dtype]
    if dtype and t == 4096:
        assert pwq.gated_workspace_size(t, rows, n, kind, exact=True) < pwq.gated_workspace_size(t, rows, n, kind)
        assert pwq.linear_backward_workspace_size(t, rows, n, kind, exact=True) < pwq.linear_backward_workspace_size(t, rows, n, kind)


def test_no_tokens(lib):  # noqa: F811
    assert back(lib, t=0, D=None, X=None, ws=None) == pwq.GPTQ_OK
    assert gated(lib, t=0, X=None, Y=None, ws=None) == pwq.GPTQ_OK
    assert gated(lib, True, t=0, X=None, Y=None, D=None, ws=None) == pwq.GPTQ_OK


@pytest.mark.parametrize("seed", range(200))
def test_any_overlap(lib, seed):  # noqa: F811
    """dX anywhere around dY, and Y around X: refused exactly where a byte is shared."""
    r = random.Random(seed)
    t, rows, n, dtype = r.choice([1, 2, 3, 7]), r.choice([1, 5, 16, 40]), r.choice([32, 64]), r.choice([0, 1])
    es = 4 if dtype == 0 else 2
    ldd = rows + r.randrange(60)
    ldx = ldd if r.random() < 0.5 and ldd >= n else n + r.randrange(60)
    X = addr(0) + es * r.randrange(-t * ldx, t * ldd + 1)
    shared = bytes_of(addr(0), ldd, t, rows, es) & bytes_of(X, ldx, t, n, es)
    got = back(lib, t=t, rows=rows, n=n, dtype=dtype, ldd=ldd, ldx=ldx, X=X)
    assert (got == pwq.GPTQ_EINVAL) == bool(shared)
    got = gated(lib, True, t=t, rows=rows, n=n, dtype=dtype, D=addr(0), X=addr(8), ldd=ldd, ldy=ldx, Y=X)
    assert (got == pwq.GPTQ_EINVAL) == bool(shared)
    ldi, ldy = n + 8 * r.randrange(9), rows + r.randrange(60)
    Y = addr(0) + es * r.randrange(-t * ldy, t * ldi + 1)
    shared = bytes_of(addr(0), ldi, t, n, es) & bytes_of(Y, ldy, t, rows, es)
    got = gated(lib, t=t, rows=rows, n=n, dtype=dtype, ldx=ldi, ldy=ldy, Y=Y)
    assert (got == pwq.GPTQ_EINVAL) == bool(shared)


def test_outputs_over_other_arguments(lib):  # noqa: F811
    for k in (1, 2):
        assert back(lib, X=addr(k)) == pwq.GPTQ_EINVAL
    assert back(lib, X=addr(4)) == pwq.GPTQ_EINVAL and back(lib, ws=addr(0)) == pwq.GPTQ_EINVAL and back(lib, ws=addr(1)) == pwq.GPTQ_EINVAL
    for backward in (False, True):
        for k in (0, 1, 2, 3, 4, 5, 6) + ((8,) if backward else ()):
            assert gated(lib, backward, Y=addr(k)) == pwq.GPTQ_EINVAL
            big = dict(t=400, rows=5120, n=4096)
            assert gated(lib, backward, **big, ws=addr(k)) == pwq.GPTQ_EINVAL
        assert gated(lib, backward, **big, Y=addr(9)) == pwq.GPTQ_EINVAL
        # Both matrices may be one, and biases too.
        assert gated(lib, backward, u=addr(1), us=addr(2), ub=addr(3)) == pwq.GPTQ_OK, pwq.check_message()


def rotary(lib, tensors=None, **kw):
    d = dict(dtype=1, rows=5, dim=96, part=64, layout=0, position=addr(8), freq=addr(9), factor=1.0, backward=0, count=None)
    d.update(kw)
    tensors = [dict()] if tensors is None else tensors
    packed = b""
    for i, t in enumerate(tensors):
        x = dict(X=addr(2 * i), ldx=None, ldxh=d["dim"], Y=addr(2 * i + 1), ldy=None, ldyh=d["dim"], heads=3)
        x.update(t)
        x["ldx"] = x["heads"] * d["dim"] if x["ldx"] is None else x["ldx"]
        x["ldy"] = x["heads"] * d["dim"] if x["ldy"] is None else x["ldy"]
        packed += pwq._ROTATED(x["X"] or 0, x["ldx"], x["ldxh"], x["Y"] or 0, x["ldy"], x["ldyh"], x["heads"], 0)
    with pwq.check_mode():
        return lib.gptq_rotary(packed, len(tensors) if d["count"] is None else d["count"], d["dtype"], d["rows"], d["dim"], d["part"],
                               d["layout"], d["position"], d["freq"], d["factor"], d["backward"], None)


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rows,dim,part", [(1, 2, 2), (5, 96, 64), (20000, 128, 128), (3, 2048, 2048), (1000, 81, 80), (1 << 23, 64, 2)])
def test_rotary_schedules(lib, dtype, layout, rows, dim, part):  # noqa: F811
    s = dict(dtype=dtype, layout=layout, rows=rows, dim=dim, part=part)
    assert rotary(lib, **s) == pwq.GPTQ_OK, pwq.check_message()
    assert rotary(lib, [dict(heads=7), dict(heads=1, ldx=dim + 3)], **s) == pwq.GPTQ_OK, pwq.check_message()
    assert rotary(lib, [dict(Y=addr(0))], **s) == pwq.GPTQ_OK, pwq.check_message()
    assert rotary(lib, [dict(ldx=dim, ldxh=rows * dim)], **s) == pwq.GPTQ_OK, pwq.check_message()


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(rows=-1), dict(rows=(1 << 23) + 1), dict(dim=1, part=2), dict(dim=2050), dict(part=0),
                                 dict(part=3), dict(part=98), dict(layout=2), dict(layout=-1), dict(position=None), dict(freq=None),
                                 dict(position=addr(8) + 2), dict(freq=addr(9) + 4), dict(factor=float("inf")), dict(factor=float("nan")),
                                 dict(count=0), dict(count=5)])
def test_rotary_refuses(lib, bad):  # noqa: F811
    assert rotary(lib, [dict()] * 5 if bad.get("count") == 5 else None, **bad) == pwq.GPTQ_EINVAL


def test_rotary_refuses_tensors(lib):  # noqa: F811
    row = 3 * 96 * 2
    for bad in (dict(X=None), dict(Y=None), dict(X=addr(0) + 1), dict(heads=0), dict(heads=65536), dict(ldx=95), dict(ldxh=95), dict(ldy=200),
                dict(Y=addr(0) + 2), dict(Y=addr(0), ldy=300), dict(Y=addr(0) + row), dict(Y=addr(8)), dict(Y=addr(9))):
        assert rotary(lib, [bad]) == pwq.GPTQ_EINVAL, bad
    assert rotary(lib, [dict(heads=65535)] * 2, dim=2048) == pwq.GPTQ_EINVAL
    # Outputs over the other tensor, and slices of one projection in place.
    assert rotary(lib, [dict(), dict(Y=addr(0))]) == pwq.GPTQ_EINVAL
    assert rotary(lib, [dict(), dict(Y=addr(1))]) == pwq.GPTQ_EINVAL
    wide = dict(ldx=9 * 96, ldy=9 * 96)
    q, k = dict(X=addr(0), Y=addr(0), **wide), dict(X=addr(0) + row, Y=addr(0) + row, **wide)
    assert rotary(lib, [q, k]) == pwq.GPTQ_OK, pwq.check_message()
    assert rotary(lib, [q, dict(k, X=addr(0) + row - 2, Y=addr(0) + row - 2)]) == pwq.GPTQ_EINVAL
    assert rotary(lib, [dict(X=None, Y=None)], rows=0, position=None, freq=None) == pwq.GPTQ_OK


def score(lib, c, b, **kw):
    d = dict(Q=addr(8), qh=2 * c.heads, dtype=1, scale=0.1, window=0, sinks=0, lse=addr(10), old=addr(11), out=addr(12))
    d.update(kw)
    d.setdefault("ldq", d["qh"] * c.dim)
    d.setdefault("ldqh", c.dim)
    with pwq.check_mode():
        return lib.gptq_cache_score(raw(c), raw(b), d["Q"], d["ldq"], d["ldqh"], d["qh"], d["dtype"], d["scale"], d["window"], d["sinks"],
                                    d["lse"], d["old"], d["out"], None)


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_score_schedules(lib, dtype, dim):  # noqa: F811
    for c, b in ((cache(dim=dim), batch()), (cache(dim=dim, page=1024, pages=3000), batch(width=1 << 16, seqs=4, rows=4, start=None)),
                 (cache(dim=dim), batch(rows=0)), (cache(dim=dim, pages=1 << 20, heads=64), batch(seqs=1 << 20, rows=3, width=9))):
        assert score(lib, c, b, dtype=dtype) == pwq.GPTQ_OK, pwq.check_message()
        assert score(lib, c, b, dtype=dtype, out=addr(11), window=5, sinks=2) == pwq.GPTQ_OK, pwq.check_message()


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(qh=4), dict(qh=0), dict(qh=3 * 65), dict(scale=float("nan")), dict(window=-1),
                                 dict(sinks=-1), dict(Q=None), dict(lse=None), dict(old=None), dict(out=None), dict(Q=addr(8) + 8),
                                 dict(lse=addr(10) + 2), dict(out=addr(12) + 1), dict(ldq=100), dict(out=addr(11) + 4), dict(out=addr(10)),
                                 dict(out=addr(8)), dict(out=addr(0)), dict(out=addr(3))])
def test_score_refuses(lib, bad):  # noqa: F811
    assert score(lib, cache(), batch(), **bad) == pwq.GPTQ_EINVAL


@pytest.mark.parametrize("which", ["table", "len", "start"])
def test_score_keeps_off_the_batch(lib, which):  # noqa: F811
    at = {"table": addr(4), "len": addr(5), "start": addr(6)}[which]
    assert score(lib, cache(), batch(**{which: at}), out=at) == pwq.GPTQ_EINVAL


def evict(lib, c, b, **kw):
    d = dict(score=addr(8), keep=50, sinks=2, recent=10, into=None, wide=0, length=addr(9), index=addr(10))
    d.update(kw)
    with pwq.check_mode():
        return lib.gptq_cache_evict(raw(c), raw(b), d["score"], d["keep"], d["sinks"], d["recent"], d["into"], d["wide"], d["length"],
                                    d["index"], None)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_evict_schedules(lib, dim):  # noqa: F811
    for b in (batch(), batch(start=None, rows=0), batch(seqs=70000), batch(rows=-5)):
        assert evict(lib, cache(dim=dim), b) == pwq.GPTQ_OK, pwq.check_message()
        assert evict(lib, cache(dim=dim), b, into=addr(11), wide=4, keep=12) == pwq.GPTQ_OK, pwq.check_message()


@pytest.mark.parametrize("bad", [dict(score=None), dict(length=None), dict(index=None), dict(keep=0), dict(keep=11), dict(keep=(1 << 30) + 1),
                                 dict(sinks=-1), dict(recent=-1), dict(score=addr(8) + 1), dict(index=addr(10) + 2), dict(length=addr(9) + 1),
                                 dict(into=addr(11), wide=0), dict(into=addr(11) + 1, wide=4), dict(into=addr(11), wide=1 << 27),
                                 dict(length=addr(5)), dict(index=addr(4)), dict(index=addr(9)), dict(length=addr(8)), dict(score=addr(1)),
                                 dict(index=addr(2)), dict(into=addr(11), wide=4, index=addr(11)), dict(into=addr(11), wide=4, length=addr(11))])
def test_evict_refuses(lib, bad):  # noqa: F811
    assert evict(lib, cache(), batch(), **bad) == pwq.GPTQ_EINVAL


def test_evict_launches_stay_below_2_32_threads(lib):  # noqa: F811
    c = cache(heads=64, pages=1 << 16)
    assert evict(lib, c, batch(seqs=(1 << 16) - 1, start=None, rows=0), keep=12) == pwq.GPTQ_OK, pwq.check_message()
    assert evict(lib, c, batch(seqs=1 << 16, start=None, rows=0), keep=12) == pwq.GPTQ_EINVAL


def test_bad_caches_and_batches(lib):  # noqa: F811
    for c in (cache(k=None), cache(dim=96), cache(page=8), cache(heads=0), cache(pages=0), cache(k_scale=addr(2) + 8)):
        assert score(lib, c, batch(), qh=6, ldq=6 * 128, ldqh=128) == pwq.GPTQ_EINVAL
        assert evict(lib, c, batch()) == pwq.GPTQ_EINVAL
    for b in (batch(table=None), batch(len=None), batch(seqs=0), batch(width=0), batch(len=addr(5) + 2), batch(width=1 << 24)):
        c = cache(page=128)
        assert score(lib, c, b) == pwq.GPTQ_EINVAL
        assert evict(lib, c, b) == pwq.GPTQ_EINVAL
    assert score(lib, cache(), batch(start=None, rows=4)) == pwq.GPTQ_EINVAL


def test_python_refusals():
    """Before any launch: gradients, kinds of tensors."""
    x = torch.zeros(2, 64, requires_grad=True)
    pair = (torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 2))
    planes = tuple(torch.zeros(1, 1, 16, 32, dtype=torch.uint8) for _ in range(4))
    h, table, length = x.view(2, 1, 64), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    z, p, f = x.detach(), torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    calls = [lambda: pwq.gptq_linear_backward(x, *pair), lambda: pwq.gptq_gated(x, pair, pair),
             lambda: pwq.gptq_gated(z, pair, pair, gate_bias=x[0, :3]), lambda: pwq.gptq_gated_backward(x, z, pair, pair),
             lambda: pwq.gptq_gated_backward(z, x, pair, pair), lambda: pwq.gptq_rotary(h, p, f),
             lambda: pwq.gptq_rotary(h.detach(), p, f, K=h), lambda: pwq.gptq_cache_score(planes, h, z, z, table, length),
             lambda: pwq.gptq_cache_evict(planes, table, length, h, 4)]
    for call in calls:
        with pytest.raises(ValueError, match="no gradient"):
            call()
    with torch.no_grad():
        for call in calls:
            with pytest.raises(ValueError) as e:
                call()
            assert "no gradient" not in str(e.value)
