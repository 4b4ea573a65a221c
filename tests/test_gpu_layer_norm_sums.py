"""GPU: the sums of dweight and dbias over many rows whose terms have one sign, where 32-bit sums lose digits with their
length.

Bounds.  With u = 2^-24: a term dy xh has two roundings, of x - mean and of its product with rstd; sums are formed in 64
bits and rounded when a lane leaves its own, when a workgroup does, and at the end, each by u of a sum that is at most
the terms' absolute values: 3 u of these for dbias and 5 u for dweight, at any number of rows (2^20 roundings of 64 bits
are 2^-33).  One u more is allowed."""
import pytest
import torch

from scale_gla_layer_amd.config import LayerNormConfig
from tests.gpu_cases import say
from tests.test_gpu_layer_norm import TYPE

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("kind", ["equal", "spread", "as x"])
@pytest.mark.parametrize("B,L,D,dtype", [
    (1, (1 << 20) + 77, 64, "f32"), (3, 70001, 333, "bf16"), (1, (1 << 18) + 5, 1001, "f32"), (2, 66000, 1024, "bf16"),
    (1, (1 << 17) + 77, 2048, "f32"), (1, (1 << 17) + 1, 4096, "bf16"), (1, 32768 + 77, 4096, "f32"), (5, 20011, 8192, "bf16"),
    (1, (1 << 16) + 77, 9000, "f32"), (1, 100003, 8200, "bf16")])
def test_terms_of_one_sign(B, L, D, dtype, kind):
    from scale_gla_layer_amd.runner import DeviceLayerNorm
    say(f"layer norm sums B={B} L={L} D={D} {dtype} {kind}")
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.empty((B, L, D), dtype=TYPE[dtype], device="cuda").normal_(generator=g)
    if kind == "as x":  # dy xh has one sign
        dy = x.clone()
    else:  # dy has
        dy = torch.full_like(x, 1e-3) if kind == "equal" else torch.empty_like(x).uniform_(0.5, 1.5, generator=g)
    op = DeviceLayerNorm(LayerNormConfig(D, dtype=dtype))
    w, b = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    y, mean, rstd = op.forward(x, w, b)
    _, dw, db = op.backward(x, dy, mean, rstd, w, b, dx=y)
    want = torch.zeros((4, D), dtype=torch.float64, device="cuda")
    for seq in range(B):
        for i in range(0, L, 8192):
            at = slice(i, i + 8192)
            t = dy[seq, at].double()
            want[1] += t.sum(0)
            want[3] += t.abs().sum(0)
            t *= (x[seq, at].double() - mean[seq, at, None].double()) * rstd[seq, at, None].double()
            want[0] += t.sum(0)
            want[2] += t.abs().sum(0)
    for name, got, value, size, n in (("dweight", dw, want[0], want[2], 6), ("dbias", db, want[1], want[3], 4)):
        worst = float(((got.double() - value).abs() / (n * U * size)).max())
        assert worst <= 1, f"{name}: {worst:.2f} of its bound"
        say(f"{name}: {worst:.2f} of its bound")
