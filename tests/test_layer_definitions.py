"""The definitions that the layer's further operators are tested against: their gradients by automatic
differentiation and by differences, in 64 bits on the CPU, and the frequencies of rotary positions."""
import math

import pytest
import torch

import layer
import operands as ref
import post_weight_quantization_amd as pwq

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def weights(rows, n, codec, g):
    return (torch.randint(0, 256, (rows, n // (2 if codec == "q4tp" else 4)), generator=g, dtype=torch.uint8),
            torch.exp2(torch.randn(rows, n // 32, generator=g) * 0.5 - 4.0))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("codec", ["q4tp", "q2tp"])
def test_gated_gradient(act, codec):
    g = torch.Generator().manual_seed(1)
    gate, up = weights(7, 64, codec, g), weights(7, 64, codec, g)
    bias = [torch.randn(7, generator=g), None]
    x, dy = torch.randn(5, 64, generator=g), torch.randn(5, 7, generator=g)
    want, _ = layer.gated_backward(dy, x, gate, up, codec, act, bias)

    def f(z):
        a = z @ ref.weight_values(*gate, codec).t() + bias[0].double()
        return ref.activate(a, act) * (z @ ref.weight_values(*up, codec).t())

    z = x.double().requires_grad_()
    assert torch.allclose(torch.autograd.grad(f(z), z, dy.double())[0], want, rtol=1e-10, atol=1e-12)
    v = torch.randn(5, 64, generator=g, dtype=torch.float64)
    h = 1e-6
    z = z.detach()
    diff = ((f(z + h * v) - f(z - h * v)) * dy).sum() / (2 * h)
    assert abs(float(diff - (want * v).sum())) < 1e-7 * float((want * v).abs().sum() + 1)


def test_slopes_bound_what_the_bounds_say():
    a = torch.linspace(-30, 30, 600001, dtype=torch.float64)
    for act in ACTS:
        k = layer.slope(a, act)
        assert float(k.abs().max()) < 1.13 and float((ref.activate(a, act).abs() - a.abs()).max()) <= 1e-12
        if act not in ("none", "relu"):
            assert float(((k[1:] - k[:-1]) / (a[1:] - a[:-1])).abs().max()) < 1.1


def test_rotary_backward_is_the_transpose():
    g = torch.Generator().manual_seed(2)
    x, y = torch.randn(4, 2, 12, generator=g), torch.randn(4, 2, 12, generator=g)
    p, f = torch.tensor([0, 5, -7, 100000]), torch.rand(5, generator=g, dtype=torch.float64)
    for layout in ("half", "interleaved"):
        a, _ = layer.rotary(x, p, f, layout, 1.3, False)
        b, _ = layer.rotary(y, p, f, layout, 1.3, True)
        assert abs(float((a[..., :10] * y[..., :10].double()).sum() - (x[..., :10].double() * b[..., :10]).sum())) < 1e-12


def test_frequencies():
    f, k = pwq.rotary_frequencies(8, device="cpu")
    assert k == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.allclose(pwq.rotary_frequencies(8, scaling="linear", stretch=4.0, device="cpu")[0], f / 4)
    b, _ = pwq.rotary_frequencies(8, scaling="base", stretch=4.0, device="cpu")
    assert math.isclose(b[0], 1.0) and math.isclose(b[3], f[3] / 4)
    r, k = pwq.rotary_frequencies(128, scaling="ramp", stretch=8.0, trained=4096, device="cpu")
    f, _ = pwq.rotary_frequencies(128, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(r[turns >= 32], f[turns >= 32]) and torch.allclose(r[turns <= 1], f[turns <= 1] / 8)
    inside = (turns > 1) & (turns < 32)
    assert inside.sum() > 5 and (r[inside] < f[inside]).all() and (r[inside] > f[inside] / 8).all()
    assert math.isclose(k, 0.1 * math.log(8) + 1)
    for bad in (dict(part=7), dict(part=0), dict(part=8, base=0.0), dict(part=8, stretch=0.5), dict(part=8, scaling="other"),
                dict(part=2, scaling="base", stretch=2.0), dict(part=8, slow=2.0, fast=2.0), dict(part=8, trained=0)):
        with pytest.raises(ValueError):
            pwq.rotary_frequencies(device="cpu", **bad)


def test_eviction_order():
    c = ref.Cache(3, 16, 1, 64)
    import numpy as np
    z = np.zeros((3, 1, 16), np.float32)
    z[2, 0] = [5, 1, 1, 9, 1, np.nan, -3, 0, -0.0, 2, 2, 2, 7, 7, 1, 1]
    table = np.array([[2, 9]], np.int32)  # the second page is not there
    left, index = layer.evict(c, z, table, np.array([20]), 6, 1, 2)
    assert left[0] == 6 and index[0, 0].tolist() == [0, 3, 5, 12, 18, 19]
