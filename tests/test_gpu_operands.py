"""Calls of the operators on quantized operands that their other tests do not make: outputs over inputs."""
import pytest
import torch

from test_gpu_linear import make

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 40, 300])
def test_out_over_x(gpu, t):
    """A square layer into its own input raises and leaves it alone; into another slice of its buffer it runs."""
    X, codes, scale, _, _ = make(t, 256, 256, torch.bfloat16, "q4tp", t)
    keep = X.clone()
    with pytest.raises(gpu.GptqError):
        gpu.gptq_linear(X, codes, scale, out=X)
    assert torch.equal(X, keep)
    both = torch.zeros(t, 512, dtype=X.dtype, device="cuda")
    both[:, 256:] = X
    gpu.gptq_linear(both[:, 256:], codes, scale, out=both[:, :256])
    assert torch.equal(both[:, :256], gpu.gptq_linear(X, codes, scale)) and torch.equal(both[:, 256:], X)


@pytest.mark.gpu
def test_gradients_are_refused_not_dropped(gpu):
    X, codes, scale, bias, _ = make(3, 40, 64, torch.float32, "q4tp", 1)
    want = gpu.gptq_linear(X, codes, scale, bias=bias)
    for kw in (dict(X=X.clone().requires_grad_()), dict(bias=bias.clone().requires_grad_()), dict(scale=scale.clone().requires_grad_())):
        args = dict(X=X, codes=codes, scale=scale, bias=bias)
        args.update(kw)
        with pytest.raises(ValueError):
            gpu.gptq_linear(**args)
        with torch.no_grad():
            assert torch.equal(gpu.gptq_linear(**args), want)
