"""Which kernels the GPU tests' sizes take, on the host: every one of them, cut and uncut."""
import ctypes

import pytest

import post_weight_quantization_amd as pwq
from test_gpu_gated import DENSE, LARGE, SMALL


def plans(t, rows, n, dtype):
    lib, p = pwq.load(), (ctypes.c_int64 * 3)()
    assert lib.gptq_check_backward_plan(dtype, t, rows, n, p) == 0
    out = [tuple(p)]
    for back in (0, 1):
        assert lib.gptq_check_gated_plan(dtype, t, rows, n, back, p) == 0
        out.append(tuple(p))
    return out


@pytest.mark.parametrize("dtype", [1, 2])
def test_large_sizes_decode(dtype):
    for t, rows, n in DENSE + [(1210, 2056, 2112), (1301, 2051, 2144), (1211, 2080, 2144), (1210, 2112, 2112)]:
        assert [p[0] for p in plans(t, rows, n, dtype)] == [3, 3, 3], (t, rows, n)
        assert [p[0] for p in plans(t, rows, n, 16 | dtype)] != [3, 3, 3]
        assert all(p[0] != 3 for p in plans(t, rows, n, 0))
    assert [p[0] for p in plans(17000, 520, 1056, dtype)] == [3, 3, 3]


def test_every_layout_is_tested():
    """The products on codes: tiles of tokens a wave, whole and in pieces; the sums' two kernels likewise."""
    back, gated = set(), set()
    for dtype in (0, 1, 2):
        for size in SMALL + LARGE + DENSE + [(37, 2048, 2048), (16, 1024, 2048), (333, 1024, 1024)]:
            b, f, g = plans(*size, dtype)
            back.add((b[0], b[1] > 1, b[2]))
            gated.add((f[0], f[1] > 1))
            gated.add((g[0], g[1] > 1, g[2] > 1))
    for tt in (1, 2, 3):
        assert (1, True, tt) in back and (1, False, tt) in back, (tt, back)
    assert (3, True, 0) in back and {(1, False), (2, False), (2, True), (3, True)} <= gated
    assert (3, True, True) in gated and any(g[0] < 3 and g[2] for g in gated if len(g) == 3)


def test_refusals():
    lib, p = pwq.load(), (ctypes.c_int64 * 3)()
    for args in ((3, 5, 5, 64), (1, 0, 5, 64), (1, 5, 0, 64), (1, 5, 5, 65)):
        assert lib.gptq_check_backward_plan(*args, p) == pwq.GPTQ_EINVAL
        assert lib.gptq_check_gated_plan(*args, 0, p) == pwq.GPTQ_EINVAL
    assert lib.gptq_check_backward_plan(1, 5, 5, 64, None) == pwq.GPTQ_EINVAL


@pytest.mark.parametrize("t,rows,n", [(3579, 5569, 1888), (2669, 6644, 4384), (2324, 3474, 3232), (354, 7172, 2144), (1210, 2101, 2080)])
def test_reported_pieces_are_those_that_are_taken(t, rows, n):
    """bf16 on decoded weights: the workspace holds the operands, and 256 KB of sums for each piece of a cut tile."""
    lib = pwq.load()
    up = lambda x, m: -(-x // m) * m  # noqa: E731
    sums = up(rows, 16) * 2
    held = 3 * up(4 * t, 256) + up(4 * sums, 256) + 512 + up(2 * t * up(n, 64), 256) + up(2 * up(sums, 256) * up(n, 64), 256)
    _, (kernel, pieces, _), _ = plans(t, rows, n, 1)
    tiles = -(-sums // 256) * -(-t // 256)
    assert kernel == 3
    assert lib.gptq_gated_workspace_size(1, t, rows, n) - held == (tiles % 256 * pieces << 18 if pieces > 1 else 0)
