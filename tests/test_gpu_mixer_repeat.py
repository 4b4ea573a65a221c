"""GPU: the gradients of linear and window attention at sizes that fill the card, again and again beside work on another
stream: the same bits every time."""
import pytest
import torch

from scale_gla_layer_amd.config import LayerNormConfig, LinearAttentionConfig, WindowAttentionConfig
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu


def _repeat(run):
    first, side = [t.clone() for t in run()], torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(side):
            x @ x
        assert all(torch.equal(a, b) for a, b in zip(run(), first)), i
    torch.cuda.synchronize()


def _random(*shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def test_linear_gradient():
    from scale_gla_layer_amd.runner import DeviceLinearAttention
    say("linear gradient, again and again")
    op = DeviceLinearAttention(LinearAttentionConfig(4, 128, 256))
    q, k, v, do = (_random(8, 2048, 4, d) for d in (128, 128, 256, 256))
    ld = torch.tensor([-0.2, -0.05, -0.01, -0.001], device="cuda")
    s, ds = (_random(8, 4, 128, 256, dtype=torch.float32) for _ in range(2))
    _repeat(lambda: op.backward(q, k, v, ld, do, state_in=s, dstate_out=ds))


def test_window_gradient():
    from scale_gla_layer_amd.runner import DeviceWindowAttention
    say("window gradient, again and again")
    op = DeviceWindowAttention(WindowAttentionConfig(16, 4, 128, 128, 1024, 4))
    q, do, (k, v) = _random(2, 4096, 16, 128), _random(2, 4096, 16, 128) + 1, (_random(2, 4096, 4, 128) * c for c in (1, 2))
    out, lse = op.forward(q, k, v)
    _repeat(lambda: (*op.forward(q, k, v), *op.backward(q, k, v, out, lse, do)))


def test_norm_gradient():
    from scale_gla_layer_amd.runner import DeviceLayerNorm
    say("norm gradient, again and again")
    op, x, dy = DeviceLayerNorm(LayerNormConfig(1024)), _random(8, 2048, 1024), _random(8, 2048, 1024) * 2
    w, b = _random(1024, dtype=torch.float32), _random(1024, dtype=torch.float32)
    y, mean, rstd = op.forward(x, w, b)
    _repeat(lambda: op.backward(x, dy, mean, rstd, w, b))
