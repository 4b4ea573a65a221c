"""GPU: the gated linear recurrence over more elements than 32 bits count."""
import pytest

from scale_gla_layer_amd.config import RecurrenceConfig

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_beyond_32_bits(dtype):
    """A sequence of more than 2^31 elements: its end, from a group boundary on, is the same bits as that part
    continued from the state there."""
    import torch
    from scale_gla_layer_amd.runner import DeviceRecurrence
    cut, D = 1 << 20, 2304
    L = cut + 4096 + 77
    g = torch.Generator(device="cuda").manual_seed(51)
    T = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, z = (torch.empty((1, L, D), dtype=T, device="cuda").normal_(generator=g) for _ in range(2))
    bias, dh = torch.full((D,), 2.0, device="cuda"), torch.randn((1, D), generator=g, device="cuda")
    op = DeviceRecurrence(RecurrenceConfig(D, "norm", 16.0, dtype))
    y, h = op.forward(x, z, bias)
    _, hc = op.forward(x[:, :cut], z[:, :cut], bias)
    ye, he = op.forward(x[:, cut:], z[:, cut:], bias, h_in=hc)
    assert torch.equal(y[:, cut:], ye) and torch.equal(h, he)
    del ye
    dx, dz, _, _ = op.backward(x, z, y, bias, dh_out=dh)
    ex, ez, _, _ = op.backward(x[:, cut:], z[:, cut:], y[:, cut:], bias, h_in=hc, dh_out=dh)
    assert torch.equal(dx[:, cut:], ex) and torch.equal(dz[:, cut:], ez)
