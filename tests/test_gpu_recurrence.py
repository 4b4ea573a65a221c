"""GPU: the gated linear recurrence against the 64-bit reference, within bounds
derived there: lengths around the chunk, odd widths, masks, strided views,
states, special values, graph replays and refusals."""
import numpy as np
import pytest

from scale_gla_layer_amd.config import RecurrenceConfig
from tests import recurrence_ref as ref
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _type(dtype):
    return _torch().bfloat16 if dtype == "bf16" else _torch().float32


def _handle(cfg):
    from scale_gla_layer_amd.runner import DeviceRecurrence
    return DeviceRecurrence(cfg)


def _inputs(B, L, D, dtype, seed, mask, zshift=2.0):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(n, generator=g)  # noqa: E731
    v = {"x": r(B, L, D), "z": r(B, L, D) * 2, "dy": r(B, L, D)}
    v = {n: t.to(_type(dtype)) for n, t in v.items()}
    v.update(bias=r(D) + zshift, h_in=r(B, D), dh_out=r(B, D), mask=None)
    if mask:
        m = torch.rand((B, L), generator=g) < {"holes": 0.7, "ragged": 1.0, "empty": 1.0}[mask]
        if mask == "ragged":
            for b in range(B):
                m[b, max(1, L - b * L // B):] = False
                m[b, :min(b, L - 1)] = False
        if mask == "empty":
            m[B // 2:] = False
        v["mask"] = m.to(torch.uint8)
    return v


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _check(name, got, want, bound):
    g = _host(got)
    assert np.all(np.isfinite(g)), f"{name}: not finite"
    off = np.abs(g - want)
    worst = np.max(off / np.maximum(bound, 1e-300) * (off > 0))
    assert worst <= 1, f"{name}: {worst:.2f} of its bound"
    say(f"{name}: {worst:.2f} of its bound")


def _case(B, L, D, dtype, mode, gamma=16.0, mask=None, state=True, seed=0):
    say(f"recurrence B={B} L={L} D={D} {dtype} {mode} gamma={gamma} mask={mask} state={state}")
    cfg = RecurrenceConfig(D, mode, gamma, dtype)
    v = _inputs(B, L, D, dtype, seed, mask)
    if not state:
        v["h_in"] = v["dh_out"] = None
    d = {n: None if t is None else t.cuda() for n, t in v.items()}
    h = {n: _host(t) for n, t in v.items()}
    op = _handle(cfg)
    y, hT = op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"])
    want, bound = ref.forward(h["x"], h["z"], h["bias"], gamma, mode, h["mask"], h["h_in"], dtype)
    _check("y", y, want["y"], bound["y"])
    _check("h_out", hT, want["h_out"], bound["h_out"])
    got = op.backward(d["x"], d["z"], d["dy"], d["bias"], d["mask"], d["h_in"], d["dh_out"])
    want, bound = ref.backward(h["x"], h["z"], h["dy"], h["bias"], gamma, mode, h["mask"], h["h_in"], h["dh_out"],
                               dtype)
    for name, t in zip(("dx", "dz", "dbias", "dh_in"), got):
        if t is not None:
            _check(name, t, want[name], bound[name])


@pytest.mark.parametrize("mode", ["plain", "convex", "norm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(1, 1, 1), (2, 7, 64), (3, 64, 260), (2, 65, 256), (1, 129, 100), (2, 700, 33)])
def test_sizes(B, L, D, dtype, mode):
    _case(B, L, D, dtype, mode, seed=L)


@pytest.mark.parametrize("dtype,B,L,D,mode,mask", [
    ("f32", 2, 4500, 66, "norm", None), ("bf16", 1, 6145, 130, "convex", "holes"), ("bf16", 2, 2049, 5, "plain", "ragged"),
    ("f32", 3, 2048, 64, "convex", "ragged"), ("bf16", 40, 300, 200, "norm", "ragged")])
def test_long_sequences(dtype, B, L, D, mode, mask):
    """Several groups of chunks, the last of them of one position; states that hardly decay."""
    _case(B, L, D, dtype, mode, mask=mask, seed=L)


def test_states_in_place_over_a_long_sequence():
    torch = _torch()
    B, L, D = 2, 3000, 128
    op = _handle(RecurrenceConfig(D, "norm", 16.0, "bf16"))
    d = {n: t.cuda() for n, t in _inputs(B, L, D, "bf16", 40, "holes").items()}
    y, hT = op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"])
    for _ in range(5):
        h = d["h_in"].clone()
        y2, h2 = op.forward(d["x"], d["z"], d["bias"], d["mask"], h, h_out=h)
        assert torch.equal(y, y2) and torch.equal(hT, h)


@pytest.mark.parametrize("mask", ["holes", "ragged", "empty"])
@pytest.mark.parametrize("dtype,L,D", [("f32", 200, 68), ("bf16", 333, 64), ("bf16", 40, 7)])
def test_masks(mask, dtype, L, D):
    _case(4, L, D, dtype, "norm", mask=mask, seed=3)


@pytest.mark.parametrize("gamma", [1.0, 200.0])
def test_other_decays_without_states(gamma):
    _case(2, 500, 64, "f32", "convex", gamma, state=False, seed=4)
    _case(2, 500, 64, "bf16", "norm", gamma, state=False, seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [5, 150])
def test_views_and_what_lies_around_them(L, dtype):
    """x and z from one wide projection, gradients into one: elements outside the views stay as they were.
    Rows that do not start at even elements take another kernel, which may round differently."""
    torch = _torch()
    B, D = 2, 64
    cfg = RecurrenceConfig(D, "norm", 16.0, dtype)
    v = _inputs(B, L, D, dtype, 6, "holes")
    d = {n: t.cuda() for n, t in v.items()}
    h = {n: _host(t) for n, t in v.items()}
    want, bound = ref.forward(h["x"], h["z"], h["bias"], 16.0, "norm", h["mask"], h["h_in"], dtype)
    gwant, gbound = ref.backward(h["x"], h["z"], h["dy"], h["bias"], 16.0, "norm", h["mask"], h["h_in"], h["dh_out"],
                                 dtype)
    op = _handle(cfg)
    plain = op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"])
    grads = op.backward(d["x"], d["z"], d["dy"], d["bias"], d["mask"], d["h_in"], d["dh_out"])
    for lead in (8, 3):
        wide = torch.full((B, L + 1, 2 * D + 16), float("nan"), dtype=_type(dtype), device="cuda")
        xs, zs = wide[:, :L, lead:lead + D], wide[:, :L, lead + D:lead + 2 * D]
        xs.copy_(d["x"])
        zs.copy_(d["z"])
        out = torch.full_like(wide, 7.0)
        state = d["h_in"].clone()
        y, hT = op.forward(xs, zs, d["bias"], d["mask"], state, y=out[:, :L, lead:lead + D], h_out=state)
        assert hT is state
        _check("y", y, want["y"], bound["y"])
        _check("h_out", hT, want["h_out"], bound["h_out"])
        if lead % 2 == 0:
            assert torch.equal(y, plain[0]) and torch.equal(hT, plain[1])
        y.fill_(7.0)
        assert bool((out == 7.0).all())
        g = torch.full_like(wide, 7.0)
        dx, dz = g[:, :L, lead:lead + D], g[:, :L, lead + D:lead + 2 * D]
        got = op.backward(xs, zs, d["dy"], d["bias"], d["mask"], d["h_in"], d["dh_out"], dx=dx, dz=dz)
        for name, a, b in zip(("dx", "dz", "dbias", "dh_in"), got, grads):
            _check(name, a, gwant[name], gbound[name])
            if lead % 2 == 0:
                assert torch.equal(a, b)
        dx.fill_(7.0)
        dz.fill_(7.0)
        assert bool((g == 7.0).all())
        # a sequence-major layout [L, B, D]
        xt, zt = d["x"].transpose(0, 1).contiguous(), d["z"].transpose(0, 1).contiguous()
        y2, _ = op.forward(xt.transpose(0, 1), zt.transpose(0, 1), d["bias"], d["mask"], d["h_in"])
        assert torch.equal(y2, plain[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["plain", "convex", "norm"])
def test_steps_continue_a_forward(mode, dtype):
    torch = _torch()
    B, L, D = 3, 90, 100
    cfg = RecurrenceConfig(D, mode, 16.0, dtype)
    v = _inputs(B, L, D, dtype, 8, "holes")
    d = {n: t.cuda() for n, t in v.items()}
    op = _handle(cfg)
    h = {n: _host(t) for n, t in v.items()}
    want, bound = ref.forward(h["x"], h["z"], h["bias"], 16.0, mode, h["mask"], h["h_in"], dtype)
    cut = 70
    y, state = op.forward(d["x"][:, :cut], d["z"][:, :cut], d["bias"], d["mask"][:, :cut].contiguous(), d["h_in"])
    ys = [y]
    for t in range(cut, L):
        yt, state = op.step(d["x"][:, t], d["z"][:, t], state, d["bias"], d["mask"][:, t].contiguous())
        ys.append(yt[:, None])
    _check("y", torch.cat(ys, 1), want["y"], bound["y"])
    _check("state", state, want["h_out"], bound["h_out"])


def test_padding_has_no_influence():
    torch = _torch()
    B, L, D = 2, 150, 64
    op = _handle(RecurrenceConfig(D, "norm", 16.0, "bf16"))
    v = _inputs(B, L, D, "bf16", 9, "holes")
    d = {n: t.cuda() for n, t in v.items()}
    off = d["mask"] == 0
    clean = [op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"]),
             op.backward(d["x"], d["z"], d["dy"], d["bias"], d["mask"], d["h_in"], d["dh_out"])]
    for value in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min):
        for n in ("x", "z", "dy"):
            d[n][off] = value
        dirty = [op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"]),
                 op.backward(d["x"], d["z"], d["dy"], d["bias"], d["mask"], d["h_in"], d["dh_out"])]
        for a, b in zip(clean, dirty):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert bool((clean[0][0][off] == 0).all()) and bool((clean[1][0][off] == 0).all())
    assert bool((clean[1][1][off] == 0).all())


@pytest.mark.parametrize("mode", ["plain", "convex", "norm"])
def test_gates_at_their_ends(mode):
    """An open gate (alpha 1), a closed one (alpha 0), and a NaN that stays in its channel from its position on."""
    torch = _torch()
    D, L = 8, 100
    op = _handle(RecurrenceConfig(D, mode, 16.0, "f32"))
    x = torch.ones(1, L, D, device="cuda")
    z = torch.zeros(1, L, D, device="cuda")
    z[..., 0], z[..., 1], z[0, 70, 2] = float("inf"), -float("inf"), float("nan")
    z[..., 3], z[..., 4] = 1e30, -1e30
    h0 = torch.full((1, D), 3.0, device="cuda")
    y, hT = op.forward(x, z, h_in=h0)
    t = torch.arange(1, L + 1, device="cuda").float()
    opened = 3.0 + t if mode == "plain" else torch.full_like(t, 3.0)
    for c in (0, 3):
        assert torch.equal(y[0, :, c], opened)
    for c in (1, 4):
        assert torch.equal(y[0, :, c], torch.ones_like(t))
    assert bool(y[0, :70, 2].isfinite().all()) and bool(y[0, 70:, 2].isnan().all()) and bool(hT[0, 2].isnan())
    assert bool(y[0, :, 5:].isfinite().all())
    dx, dz, _, dh = op.backward(x, z, torch.ones_like(x), h_in=h0)
    for c in (0, 1, 3, 4):
        assert torch.equal(dz[0, :, c], torch.zeros(L, device="cuda"))
        assert bool(dx[0, :, c].isfinite().all())
    assert torch.equal(dh[0, 0], torch.tensor(float(L), device="cuda")) and dh[0, 1] == 0


@pytest.mark.parametrize("L", [40, 300])
def test_gradient_of_the_state_alone_and_repeated_calls(L):
    torch = _torch()
    B, D = 2, 64
    op = _handle(RecurrenceConfig(D, "convex", 16.0, "f32"))
    d = {n: t.cuda() for n, t in _inputs(B, L, D, "f32", 11, None).items() if t is not None}
    zero = torch.zeros_like(d["x"])
    a = op.backward(d["x"], d["z"], None, d["bias"], None, d["h_in"], d["dh_out"])
    b = op.backward(d["x"], d["z"], zero, d["bias"], None, d["h_in"], d["dh_out"])
    c = op.backward(d["x"], d["z"], zero, d["bias"], None, d["h_in"], d["dh_out"])
    for s, t, u in zip(a, b, c):
        assert torch.equal(s, t) and torch.equal(t, u)


def test_captured_calls_share_nothing():
    """Two graphs and eager calls in turn, each replay against the eager result."""
    torch = _torch()
    B, L, D = 2, 300, 128
    op = _handle(RecurrenceConfig(D, "norm", 16.0, "bf16"))
    sets = []
    for seed in (20, 21):
        d = {n: t.cuda() for n, t in _inputs(B, L, D, "bf16", seed, "holes").items()}
        call = lambda d=d: (*op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"]),  # noqa: E731
                            *op.backward(d["x"], d["z"], d["dy"], d["bias"], d["mask"], d["h_in"], d["dh_out"]))
        eager = call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        sets.append((graph, out, eager, call))
    for _ in range(3):
        for graph, out, eager, call in sets:
            for t in out:
                t.zero_()
            graph.replay()
            assert all(torch.equal(s, t) for s, t in zip(call(), eager))
            torch.cuda.synchronize()
            assert all(torch.equal(s, t) for s, t in zip(out, eager))


def test_another_stream():
    torch = _torch()
    B, L, D = 2, 500, 256
    op = _handle(RecurrenceConfig(D, "norm", 16.0, "bf16"))
    d = {n: t.cuda() for n, t in _inputs(B, L, D, "bf16", 12, "holes").items()}
    want = op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(side):
            got.append(op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"]))
        got.append(op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"]))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


@pytest.mark.parametrize("L,D", [(5, 64), (700, 96), (2000, 130)])
def test_two_streams_at_once(L, D):
    """Training passes of different inputs, interleaved on two streams, against each alone."""
    torch = _torch()
    op = _handle(RecurrenceConfig(D, "norm", 16.0, "f32"))
    sets = [{n: t.cuda() for n, t in _inputs(3, L, D, "f32", seed, "holes").items()} for seed in (30, 31)]

    def call(d):
        y, h = op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"])
        return [y, h, *op.backward(d["x"], d["z"], d["x"], d["bias"], d["mask"], d["h_in"], h)]

    want = [call(d) for d in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for _ in range(5):
        for s, d, w in zip(streams, sets, want):
            with torch.cuda.stream(s):
                got.append((call(d), w))
    torch.cuda.synchronize()
    for g, w in got:
        assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("gamma", [1e-6, 1e6])
@pytest.mark.parametrize("mode", ["plain", "convex", "norm"])
def test_the_ends_of_the_normalizers_range(gamma, mode):
    """Gates that forget all, or nothing: results and gradients are numbers."""
    torch = _torch()
    op = _handle(RecurrenceConfig(64, mode, gamma, "f32"))
    d = {n: t.cuda() for n, t in _inputs(2, 300, 64, "f32", 32, "holes").items()}
    y, h = op.forward(d["x"], d["z"], d["bias"], d["mask"], d["h_in"])
    for t in (y, h, *op.backward(d["x"], d["z"], d["x"], d["bias"], d["mask"], d["h_in"], h)):
        assert bool(t.isfinite().all())


def test_refusals():
    torch = _torch()
    op = _handle(RecurrenceConfig(64, "norm", 16.0, "bf16"))
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    h = torch.zeros(2, 64, device="cuda")
    bad = [dict(x=x.float()), dict(z=x[:, :7]), dict(z=x.cpu()), dict(bias=torch.zeros(63, device="cuda")),
           dict(bias=torch.zeros(64, dtype=torch.bfloat16, device="cuda")), dict(h_in=h[:1]),
           dict(mask=torch.ones(2, 8, device="cuda")), dict(mask=torch.ones(2, 7, dtype=torch.uint8, device="cuda")),
           dict(x=x[..., ::2].repeat(1, 1, 2)[..., :32]), dict(y=x[:1].expand(2, 8, 64)),
           dict(z=torch.zeros(2, 64, 8, dtype=torch.bfloat16, device="cuda").transpose(1, 2)),
           dict(h_out=torch.zeros(64, 2, device="cuda").t())]
    for kw in bad:
        with pytest.raises(ValueError):
            op.forward(**{"x": x, "z": x, **kw})
    with pytest.raises(ValueError):
        op.step(x, x, h)
    with pytest.raises(ValueError):
        op.backward(x, x, x[:, :3])
    from scale_gla_layer_amd.binding import MsglaError
    with pytest.raises(MsglaError):
        op.backward(x, x, None)
