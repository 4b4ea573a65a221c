"""GPU: states and their gradients that are renewed in place, from one workgroup a sequence to several groups
of them: the same bits as with buffers of their own, call after call."""
import pytest

from scale_gla_layer_amd import binding
from scale_gla_layer_amd.config import RecurrenceConfig
from tests.gpu_cases import say
from tests.test_gpu_recurrence import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["plain", "norm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(3, 40, 64), (2, 100, 33), (8, 1000, 256), (2, 2048, 1024), (2, 3000, 130)])
def test_states_in_place(B, L, D, dtype, mode):
    import torch
    from scale_gla_layer_amd.runner import DeviceRecurrence
    say(f"in place B={B} L={L} D={D} {dtype} {mode}")
    cfg = RecurrenceConfig(D, mode, 16.0, dtype)
    op = DeviceRecurrence(cfg)
    d = {n: t.cuda() for n, t in _inputs(B, L, D, dtype, 50, "holes").items()}
    y, hT = op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"])
    grads = op.backward(d["x"], d["z"], d["dy"], d["bias"], d["mask"], d["h_in"], d["dh_out"])
    room = torch.empty(binding.msgla_recurrence_backward_workspace_bytes(cfg, B, L), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        h = d["h_in"].clone()
        y2, _ = op.forward(d["x"], d["z"], d["bias"], d["mask"], h, h_out=h)
        assert torch.equal(y2, y) and torch.equal(h, hT)
        dh, dx, dz, dbias = d["dh_out"].clone(), *(torch.empty_like(g) for g in grads[:3])
        binding.msgla_recurrence_backward(cfg, d["x"], d["z"], d["dy"], dx, dz, room, d["bias"], d["mask"], d["h_in"], dh,
                                          dbias, dh)
        for a, b in zip((dx, dz, dbias, dh), grads):
            assert torch.equal(a, b)
