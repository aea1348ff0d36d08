"""What the operators on quantized operands refuse in their Python calls before any launch."""
import pytest
import torch

import post_weight_quantization_amd as pwq


def calls(x, r=None):
    codes, scale = torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 2)
    planes = tuple(torch.zeros(1, 1, 16, 32, dtype=torch.uint8) for _ in range(4))
    table, length = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    h = x[:1].view(1, 1, 64)
    yield lambda: pwq.gptq_linear(x, codes, scale)
    yield lambda: pwq.gptq_linear(x.detach(), codes, scale, residual=h[0])
    yield lambda: pwq.gptq_linear(x.detach(), codes, scale, bias=h[0, 0])
    yield lambda: pwq.gptq_cache_write(planes, h, h.detach(), table, length)
    yield lambda: pwq.gptq_cache_write(planes, h.detach(), h, table, length)
    yield lambda: pwq.gptq_cache_attention(planes, h, table, length)


def test_gradients_are_refused():
    """An output without history would drop the gradient of whoever differentiates through the call."""
    x = torch.zeros(2, 64, requires_grad=True)
    for call in calls(x):
        with pytest.raises(ValueError, match="no gradient"):
            call()
    with torch.no_grad():
        for call in calls(x):
            with pytest.raises(ValueError) as e:  # host tensors, but not for their gradient
                call()
            assert "no gradient" not in str(e.value)


def test_exact_weights_without_decoding():
    """The sizes that decode the weights ask for them in the workspace, and with ``exact`` do not."""
    for kind in (torch.bfloat16, torch.float16):
        assert pwq.linear_workspace_size(4096, 5120, 17408, kind) > 2 * 5120 * 17408
        assert pwq.linear_workspace_size(4096, 5120, 17408, kind, exact=True) < 2 * 5120 * 17408
    assert pwq.linear_workspace_size(333, 2048, 8192, torch.float32, exact=True) == pwq.linear_workspace_size(333, 2048, 8192, torch.float32)
