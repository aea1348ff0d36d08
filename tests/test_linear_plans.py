"""Which kernel of gptq_linear the GPU tests' sizes take: a change of the rules that leaves a kernel, its
pieces of K or one of its epilogues without a test fails here, on the CPU."""
import ctypes

import pytest
import torch

import post_weight_quantization_amd as pwq
import test_gpu_linear
import test_gpu_linear_dense
import test_gpu_operands
import test_gpu_precision

F32, BF16, F16, EXACT = 0, 1, 2, 16


def plan(dtype, t, rows, n):
    p = (ctypes.c_int64 * 4)()
    assert pwq.load().gptq_check_linear_plan(dtype, t, rows, n, p) == pwq.GPTQ_OK
    return tuple(p)


def sizes(test, names="t,rows,n"):
    """The sizes a test is parametrised over."""
    for m in test.pytestmark:
        if m.name == "parametrize" and m.args[0].startswith(names):
            return [v[:3] for v in m.args[1]]
    raise AssertionError(f"{test.__name__} has no sizes")


def test_refuses():
    p = (ctypes.c_int64 * 4)()
    for args in ((3, 1, 1, 32), (BF16, 0, 1, 32), (BF16, 1, 0, 32), (BF16, 1, 1, 33), (32, 1, 1, 32)):
        assert pwq.load().gptq_check_linear_plan(*args, p) == pwq.GPTQ_EINVAL
    assert pwq.load().gptq_check_linear_plan(BF16, 1, 1, 32, None) == pwq.GPTQ_EINVAL


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_decoded_weights(dtype):
    whole, cut = [], []
    for t, rows, n in test_gpu_linear_dense.SIZES:
        kernel, pieces, w, c = plan(dtype, t, rows, n)
        assert kernel == 3
        whole.append(w)
        cut.append(c)
        assert (pieces > 1) == (c > 0)
    # The kernel's own epilogue alone, with rows that part Y's vectors, 16 columns of a lane, and neither.
    assert cut[:3] == [0, 0, 0] and all(w > 0 for w in whole[:3])
    rows = [r for _, r, _ in test_gpu_linear_dense.SIZES[:3]]
    assert rows[0] % 8 and rows[1] % 8 == 0 and rows[1] % 16 and rows[2] % 16 == 0
    assert whole[3] > 0 and cut[3] > 0 and whole[4] == 0 and cut[4] > 0
    # The other tests that mean this kernel.
    for t, rows, n in sizes(test_gpu_linear.test_large_products):
        assert plan(dtype, t, rows, n)[0] == 3
    assert plan(dtype, 1100, 8205, 608)[0] == 3 and (1100, 8205, 608) in sizes(test_gpu_operands.test_a_token_with_an_infinity)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_codes(dtype):
    """Each way of the codes' kernels has a size whose sums are held to the model, never decoded weights."""
    ways = set()
    for t, rows, n in sizes(test_gpu_precision.test_product):
        kernel, pieces, _, _ = plan(dtype, t, rows, n)
        assert kernel in (1, 2)
        ways.add((kernel, pieces > 1, t <= 16))
    assert ways >= {(1, False, True), (1, True, True), (1, False, False), (2, True, False)}
    assert {plan(dtype, t, rows, n)[0] for t, rows, n in sizes(test_gpu_linear.test_sizes)} == {1, 2}
    assert any(plan(dtype, t, rows, n)[:2] == (2, 1) for t, rows, n in
               sizes(test_gpu_linear.test_sizes) + sizes(test_gpu_linear.test_pieces_of_k) + sizes(test_gpu_precision.test_product))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_exact_weights_are_never_decoded(dtype):
    for t in (1, 300, 2100, 4096, 1 << 20):
        for rows, n in ((8205, 608), (5120, 17408), (100, 65536)):
            assert plan(EXACT | dtype, t, rows, n)[0] in (1, 2)
    assert plan(dtype, 4096, 5120, 17408)[0] == 3
