"""gptq_linear on decoded weights (many tokens, 16 bits) in the kernel's own epilogue and in the one behind pieces
of K: every activation, bias, residual, rows of Y that keep 16-byte vectors and rows that do not.
test_linear_plans.py states which way each size goes."""
import pytest
import torch

import operands as ref
import precision
from test_gpu_linear import make

TYPES = [torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# Whole tiles with rows past Y's alignment, past a lane's 16 columns, and neither; whole and cut; cut alone.
SIZES = [(1100, 8205, 608), (1100, 8216, 608), (1030, 8448, 640), (2600, 6213, 800), (1000, 2056, 4128)]


def sample(rows):
    """The first rows, the last ones, some between."""
    return torch.cat([torch.arange(70), torch.arange(rows - 130, rows), torch.arange(2000, 2056)]).unique()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_epilogues(gpu, kind, act, size):
    """Y alone, inside padded rows of each alignment, beside padded residuals of each; padding left alone."""
    t, rows, n = SIZES[size]
    codec = "q2tp" if size % 2 else "q4tp"
    X, codes, scale, bias, residual = make(t, rows, n, kind, codec, size)
    pick = sample(rows)
    z, sigma = precision.linear_rounded(X, codes[pick], scale[pick], codec)
    for with_bias, with_residual, pad_y, pad_r in ((0, 0, 0, 0), (1, 1, 0, 0), (1, 0, 3, 0), (0, 1, 8, 5), (1, 1, 8, 8), (1, 1, 16, 0)):
        out = torch.full((t, rows + pad_y), 3.0, dtype=kind, device="cuda")
        r = None
        if with_residual:
            r = torch.full((t, rows + pad_r), 5.0, dtype=kind, device="cuda")
            r[:, :rows] = residual
            r = r[:, :rows]
        y = gpu.gptq_linear(X, codes, scale, codec, bias if with_bias else None, act, r, out=out[:, :rows])
        w = z + (bias.double().cpu()[pick] if with_bias else 0.0)
        want = ref.activate(w, act)
        spread = 1.13 * sigma + 2.0 ** -22 * want.abs() + 2.0 ** -24 * w.abs()  # no activation is steeper than 1.13
        want = want + (residual.double().cpu()[:, pick] if with_residual else 0.0)
        ok, found = precision.holds(y[:, pick.cuda()], want, spread, kind)
        assert ok, (with_bias, with_residual, pad_y, pad_r, found)
        assert (out[:, rows:] == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_every_output(gpu, kind, size):
    """All rows and tokens of Y, in place over the residual, X's rows padded with NaN."""
    t, rows, n = SIZES[size]
    codec = "q4tp" if size % 2 else "q2tp"
    X, codes, scale, bias, residual = make(t, rows, n, kind, codec, size + 10)
    wide = torch.full((t, n + 64), float("nan"), dtype=kind, device="cuda")
    wide[:, 32:32 + n] = X
    z, sigma = precision.linear_rounded(X, codes, scale, codec)
    y = residual.clone()
    gpu.gptq_linear(wide[:, 32:32 + n], codes, scale, codec, bias, "silu", y, out=y)
    w = z + bias.double().cpu()
    want = ref.activate(w, "silu") + residual.double().cpu()
    ok, found = precision.holds(y, want, 1.13 * sigma + 2.0 ** -22 * want.abs() + 2.0 ** -24 * w.abs(), kind)
    assert ok, found


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_same_bits_on_any_stream_and_in_a_workspace_of_ones_own(gpu, kind, size):
    t, rows, n = SIZES[size]
    X, codes, scale, bias, residual = make(t, rows, n, kind, "q4tp", size)
    y = gpu.gptq_linear(X, codes, scale, "q4tp", bias, "gelu", residual)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = gpu.gptq_linear(X, codes, scale, "q4tp", bias, "gelu", residual, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, z)
    need = gpu.linear_workspace_size(t, rows, n, kind)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")   # NaN wherever it is not written first
    assert torch.equal(y, gpu.gptq_linear(X, codes, scale, "q4tp", bias, "gelu", residual, workspace=ws[:need]))
    assert (ws[need:] == 255).all()
    # Two calls at once, each with its own workspace.
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    both = [gpu.gptq_linear(X, codes, scale, "q4tp", bias, "gelu", residual, stream=q) for q in (s, other)]
    torch.cuda.synchronize()
    assert torch.equal(both[0], y) and torch.equal(both[1], y)
