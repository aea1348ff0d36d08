"""Arguments of the operators on quantized operands that share memory: what the calls refuse, against
the bytes counted one by one, and what they have to take (the residual in place, slices of one buffer)."""
import random

import pytest

import post_weight_quantization_amd as pwq
from test_operands_host import addr, attend, batch, cache, lib, linear, read  # noqa: F401


def bytes_of(p, ld, rows, cols, es):
    return {p + es * (r * ld + c) + k for r in range(rows) for c in range(cols) for k in range(es)}


def test_y_over_x(lib):  # noqa: F811
    """A square layer written over its own input, whole or by one token, and the arguments that are not X."""
    assert linear(lib, Y=addr(0), rows=96, residual=None) == pwq.GPTQ_EINVAL
    assert linear(lib, Y=addr(0) + 4 * 96 * 2, rows=96, residual=None) == pwq.GPTQ_EINVAL
    assert linear(lib, Y=addr(0) + 5 * 96 * 2, rows=96, residual=None) == pwq.GPTQ_OK
    for k in (1, 2, 3):
        assert linear(lib, Y=addr(k), residual=None) == pwq.GPTQ_EINVAL
    # Sums in pieces and decoded weights: the workspace.
    for t, rows, n in ((13, 5120, 17408), (4096, 5120, 17408)):
        assert linear(lib, t=t, rows=rows, n=n, Y=addr(6), residual=None) == pwq.GPTQ_EINVAL
        assert linear(lib, t=t, rows=rows, n=n, residual=None) == pwq.GPTQ_OK


def test_residual_in_place_or_apart(lib):  # noqa: F811
    assert linear(lib, residual=addr(5)) == pwq.GPTQ_OK
    assert linear(lib, residual=addr(5), ldr=40, ldy=40) == pwq.GPTQ_OK
    assert linear(lib, residual=addr(5), ldr=40, ldy=33) == pwq.GPTQ_EINVAL
    assert linear(lib, residual=addr(5), ldr=40, ldy=33, t=1) == pwq.GPTQ_OK
    assert linear(lib, residual=addr(5) + 2) == pwq.GPTQ_EINVAL
    assert linear(lib, residual=addr(5) + 5 * 33 * 2) == pwq.GPTQ_OK


@pytest.mark.parametrize("seed", range(300))
def test_any_overlap(lib, seed):  # noqa: F811
    """Y anywhere around X, with strides alike and not: refused exactly where a byte is shared."""
    r = random.Random(seed)
    t, rows, n, dtype = r.choice([1, 2, 3, 7]), r.choice([1, 5, 16, 40]), r.choice([32, 64]), r.choice([0, 1])
    es = 4 if dtype == 0 else 2
    ldx = n + 8 * r.randrange(12)
    ldy = ldx if r.random() < 0.5 and ldx >= rows else rows + r.randrange(60)
    Y = addr(0) + es * r.randrange(-t * ldy, t * ldx + 1)
    shared = bytes_of(addr(0), ldx, t, n, es) & bytes_of(Y, ldy, t, rows, es)
    got = linear(lib, t=t, rows=rows, n=n, dtype=dtype, ldx=ldx, ldy=ldy, Y=Y, residual=None)
    # Disjoint rows of one buffer may still meet in the schedule check's coarser ranges: only the refusal is meant.
    assert (got == pwq.GPTQ_EINVAL) == bool(shared), (t, rows, n, ldx, ldy, (Y - addr(0)) // es)


def test_attention_over_its_queries(lib):  # noqa: F811
    c, b = cache(), batch()
    assert attend(lib, c, b, O=addr(8)) == pwq.GPTQ_OK
    assert attend(lib, c, b, O=addr(8), ldo=6 * 128 + 8) == pwq.GPTQ_EINVAL
    assert attend(lib, c, b, O=addr(8), ldo=128, ldoh=11 * 128) == pwq.GPTQ_EINVAL


def test_keys_read_over_values(lib):  # noqa: F811
    assert read(lib, cache(), batch(), V=addr(8)) == pwq.GPTQ_EINVAL


def test_outputs_over_part_of_an_argument(lib):  # noqa: F811
    """Rows shared in part, slices of one projection's buffer, the cache's own planes."""
    c, b = cache(), batch()
    row = 6 * 128 * 2
    assert attend(lib, c, b, O=addr(8) + row) == pwq.GPTQ_EINVAL
    assert attend(lib, c, b, O=addr(8) + 11 * row) == pwq.GPTQ_OK
    wide = 3 * 6 * 128
    assert attend(lib, c, b, ldq=wide, ldo=wide, O=addr(8) + row) == pwq.GPTQ_OK
    assert attend(lib, c, b, ldq=wide, ldo=wide, O=addr(8) + row - 256) == pwq.GPTQ_EINVAL
    row = 3 * 128 * 2
    assert read(lib, c, b, V=addr(8) + row) == pwq.GPTQ_EINVAL
    assert read(lib, c, b, V=addr(8) + row, ld=2 * 3 * 128) == pwq.GPTQ_OK
    for plane in range(4):
        assert attend(lib, c, b, O=addr(plane)) == pwq.GPTQ_EINVAL
        assert read(lib, c, b, K=addr(plane)) == pwq.GPTQ_EINVAL
        assert read(lib, c, b, K=None, V=addr(plane)) == pwq.GPTQ_EINVAL


def test_exact_weights_schedule(lib):  # noqa: F811
    for dtype in (0, 1, 2):
        for t, rows, n in ((1, 1, 32), (4096, 5120, 17408), (333, 2048, 8192), (1 << 24, 5, 64)):
            assert linear(lib, dtype=16 | dtype, t=t, rows=rows, n=n) == pwq.GPTQ_OK, pwq.check_message()
    for dtype in (3, 32, 32 | 1, -16, -17):
        assert linear(lib, dtype=16 | dtype if dtype == 3 else dtype) == pwq.GPTQ_EINVAL
        assert lib.gptq_linear_workspace_size(16 | dtype if dtype == 3 else dtype, 5, 33, 96) == 0
