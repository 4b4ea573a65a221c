"""GPU: the recurrence where gates are all but open, so that 1 - alpha^2 is less than the least normal 32-bit
number: forward, backward and steps against the 64-bit reference.

Bounds.  To those of the reference come the absolute errors of numbers without all their bits.  exp(-(z + b)) is
0 below 2^-126, that is from z + b = 87.33 on.  1 - alpha^2 is formed by three roundings, each off by at most
2^-150, of which the first is doubled: 2^-148 in all; as beta is its square root, beta's relative error is at most
2^-148 / (1 - alpha^2) more.  sigmoid(-z - b) / gamma is off by 2^-149 more.  dz holds their product."""
import numpy as np
import pytest

from scale_gla_layer_amd.config import RecurrenceConfig
from tests import recurrence_ref as ref
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -149


def _extra(v, gamma, mode, mask):
    """Bounds of y, h_out, dx, dz beyond the reference's, for h_in, dh_out and a mask of ones."""
    zb = v["z"] + v["bias"]
    alpha, beta, slope, sig, _ = ref.gates(v["z"], v["bias"], gamma, mode)
    s = sig / gamma
    gone = zb > 87.33
    with np.errstate(all="ignore"):
        rb = np.where(gone, 1.0, 2.0 ** -148 / beta ** 2)
        assert np.all(rb[~gone] < 0.5)
        rr = np.where(gone, 1.0, rb / (1 - rb))  # of 1 / beta
        rs = np.where(gone, 1.0, LEAST / s)
    B, L, D = v["x"].shape
    h, X, ey, before, eb = v["h_in"].copy(), np.zeros((B, D)), np.zeros((B, L, D)), np.zeros((B, L, D)), np.zeros((B, L, D))
    for t in range(L):
        before[:, t], eb[:, t] = h, X
        X = alpha[:, t] * X + np.abs(beta[:, t] * v["x"][:, t]) * rb[:, t] + LEAST
        h = alpha[:, t] * h + beta[:, t] * v["x"][:, t]
        ey[:, t] = X
    c, dh = v["dh_out"].copy(), np.zeros((B, L, D))
    for t in reversed(range(L)):
        dh[:, t] = c + v["dy"][:, t]
        c = alpha[:, t] * dh[:, t]
    ex = np.abs(beta * dh) * rb + LEAST
    inner = np.abs(slope * v["x"])
    ez = np.abs(dh) * (inner * s * ((1 + rr) * (1 + rs) - 1) + (np.abs(alpha * before) * rs + eb * (1 + rs)) * s) + 4 * LEAST
    return {"y": ey, "h_out": X, "dx": ex, "dz": ez, "dbias": ez.sum((0, 1)), "dh_in": 0.0}


def _check(name, got, want, bound):
    g = got.double().cpu().numpy()
    assert np.all(np.isfinite(g)), f"{name}: not finite"
    worst = float(np.max(np.abs(g - want) / bound))
    assert worst <= 1, f"{name}: {worst:.2f} of its bound"
    say(f"{name}: {worst:.2f} of its bound")


@pytest.mark.parametrize("L", [5, 150])
@pytest.mark.parametrize("gamma", [1.0, 8.0, 16.0, 1e6])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_all_but_open(dtype, gamma, L):
    import torch
    from scale_gla_layer_amd.runner import DeviceRecurrence
    say(f"open gates {dtype} gamma={gamma} L={L}")
    D, B = 201, 2
    g = torch.Generator().manual_seed(L)
    r = lambda *n: torch.randn(n, generator=g)  # noqa: E731
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    # z + b from 70 to 90 over the channels, a little different at each position
    t = {"x": r(B, L, D).to(dt), "z": (0.25 * r(B, L, D)).clamp(-1, 1).to(dt), "dy": r(B, L, D).to(dt)}
    t.update(bias=torch.linspace(70, 90, D), h_in=1e-18 * r(B, D), dh_out=r(B, D))
    v = {n: x.double().numpy() for n, x in t.items()}
    d = {n: x.cuda() for n, x in t.items()}
    op = DeviceRecurrence(RecurrenceConfig(D, "norm", gamma, dtype))
    more = _extra(v, gamma, "norm", None)
    y, hT = op.forward(d["x"], d["z"], d["bias"], None, d["h_in"])
    want, bound = ref.forward(v["x"], v["z"], v["bias"], gamma, "norm", None, v["h_in"], dtype)
    _check("y", y, want["y"], bound["y"] + (1 + ref.HALF[dtype]) * more["y"])
    _check("h_out", hT, want["h_out"], bound["h_out"] + more["h_out"])
    h, ys = d["h_in"].clone(), []
    for i in range(L):
        yt, h = op.step(d["x"][:, i], d["z"][:, i], h, d["bias"])
        ys.append(yt)
    _check("steps' y", torch.stack(ys, 1), want["y"], bound["y"] + (1 + ref.HALF[dtype]) * more["y"])
    _check("steps' state", h, want["h_out"], bound["h_out"] + more["h_out"])
    got = op.backward(d["x"], d["z"], d["dy"], d["bias"], None, d["h_in"], d["dh_out"])
    want, bound = ref.backward(v["x"], v["z"], v["dy"], v["bias"], gamma, "norm", None, v["h_in"], v["dh_out"], dtype)
    for name, x in zip(("dx", "dz", "dbias", "dh_in"), got):
        extra = more[name] if name in ("dbias", "dh_in") else (1 + ref.HALF[dtype]) * more[name]
        _check(name, x, want[name], bound[name] + extra)
