"""GPU: linear attention with a decay per head against the 64-bit reference, within bounds derived there: lengths around
the chunk and the segments, head widths, padded batches, states, special decays, views, graph replays and refusals."""
import math

import pytest
import torch

from scale_gla_layer_amd.config import LinearAttentionConfig
from tests import linear_ref as ref
from tests.gpu_cases import say
from tests.test_gpu_layer_norm import TYPE, _dev, _f64, check

pytestmark = pytest.mark.gpu
SOME = (-0.01, -0.5, -math.inf, -1e-4, 0.0)  # log decays that heads take in turn


def _handle(cfg):
    from scale_gla_layer_amd.runner import DeviceLinearAttention
    return DeviceLinearAttention(cfg)


def _inputs(B, L, H, dk, dv, dtype, lens=None, state=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(n, generator=g)  # noqa: E731
    v = {"q": r(B, L, H, dk), "k": r(B, L, H, dk), "v": r(B, L, H, dv), "dout": r(B, L, H, dv)}
    v = {n: t.to(TYPE[dtype]) for n, t in v.items()}
    v["log_decay"] = torch.tensor([SOME[h % len(SOME)] for h in range(H)])
    v["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    v["state"], v["dstate"] = (r(B, H, dk, dv), r(B, H, dk, dv)) if state else (None, None)
    return v


def _case(B, L, H, dk, dv, dtype, lens=None, state=True, views=lambda t: t, seed=0):
    say(f"linear attention B={B} L={L} H={H} dk={dk} dv={dv} {dtype} lens={lens} state={state}")
    cfg = LinearAttentionConfig(H, dk, dv, dtype=dtype)
    h, v = _handle(cfg), _inputs(B, L, H, dk, dv, dtype, lens, state, seed)
    d = {n: _dev(t) for n, t in v.items()}
    if lens is not None:  # padding has no influence, whatever it holds
        for n in ("q", "k", "v", "dout"):
            for b, m in enumerate(lens):
                d[n][b, max(0, m):] = float("nan")
    q, k, x, do = (views(d[n]) for n in ("q", "k", "v", "dout"))
    out, last = h.forward(q, k, x, d["log_decay"], lens=d["lens"], state_in=d["state"])
    ln = [L] * B if lens is None else [min(max(n, 0), L) for n in lens]
    f = {n: _f64(t) for n, t in v.items() if n != "lens"}
    (wo, ws), (bo, bs) = ref.walk(f["q"], f["k"], f["v"], f["log_decay"], ln, f["state"], cfg.scale, dtype)
    check("out", out, wo, bo)
    check("state", last, ws, bs)
    dq, dk_, dv_, ds = h.backward(q, k, x, d["log_decay"], do, lens=d["lens"], state_in=d["state"], dstate_out=d["dstate"])
    want, bound = ref.backward(f["q"], f["k"], f["v"], f["log_decay"], ln, f["state"], f["dout"], f["dstate"], cfg.scale, dtype)
    assert (ds is None) == (not state)
    for n, t in (("dq", dq), ("dk", dk_), ("dv", dv_), ("dstate", ds)):
        if t is not None:
            check(n, t, want[n], bound[n])
    return h, d, (out, last, dq, dk_, dv_, ds)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200])
def test_lengths(L, dtype):
    _case(2, L, 3, 32, 64, dtype, state=L % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(8, 8), (64, 64), (72, 40), (80, 96), (128, 128), (128, 256), (136, 264 - 8), (256, 128),
                                   (256, 256), (24, 200)])
def test_widths(dk, dv, dtype):
    _case(1, 150, 2, dk, dv, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded(dtype):
    _case(6, 140, 2, 64, 96, dtype, lens=[140, 0, 1, 64, 65, 139])
    _case(4, 70, 5, 16, 32, dtype, lens=[-3, 500, 70, 33], state=False)


@pytest.mark.parametrize("B,L,H,dk,dv,dtype,lens", [
    (1, 1100, 2, 64, 64, "bf16", None), (1, 2500, 1, 128, 64, "f32", None), (2, 1025, 1, 32, 96, "bf16", [1025, 300]),
    (3, 4097, 1, 16, 16, "bf16", [4097, 1, 2048]), (1, 5000, 5, 64, 128, "bf16", None)])
def test_segments(B, L, H, dk, dv, dtype, lens):
    _case(B, L, H, dk, dv, dtype, lens)


def test_many_heads():
    _case(40, 70, 16, 64, 64, "bf16", state=False)


def test_strided_views():
    def packed(t):  # heads of a wider projection, positions of a longer tensor
        B, L, H, d = t.shape
        big = torch.full((B, L + 3, H, d + 24), float("nan"), dtype=t.dtype, device="cuda")
        view = big[:, 2:2 + L, :, 16:16 + d]
        view.copy_(t)
        return view
    _case(2, 100, 3, 64, 96, "bf16", views=packed)
    _case(2, 100, 3, 64, 96, "f32", views=lambda t: t.transpose(1, 2).contiguous().transpose(1, 2))


@pytest.mark.parametrize("L", [100, 1500])
def test_state_in_place_and_continued(L):
    """A sequence in two parts is the whole one, and the state may be renewed in place."""
    h, d, (out, last, *_) = _case(2, L, 2, 64, 64, "f32")
    state, m = d["state"].clone(), L // 3
    first, s1 = h.forward(*(d[n][:, :m].contiguous() for n in ("q", "k", "v")), d["log_decay"], state_in=state, state_out=state)
    second, s2 = h.forward(*(d[n][:, m:].contiguous() for n in ("q", "k", "v")), d["log_decay"], state_in=state, state_out=state)
    assert s1 is state and s2 is state
    scale = float(out.abs().max())
    assert float((torch.cat((first, second), 1) - out).abs().max()) <= 1e-4 * scale
    assert float((state - last).abs().max()) <= 1e-4 * float(last.abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 8, 8), (3, 5, 128, 256), (16, 4, 80, 40), (2, 2, 256, 104)])
def test_step(B, H, dk, dv, dtype):
    say(f"linear step B={B} H={H} dk={dk} dv={dv} {dtype}")
    cfg = LinearAttentionConfig(H, dk, dv, dtype=dtype)
    h, v = _handle(cfg), _inputs(B, 1, H, dk, dv, dtype)
    d, f = {n: _dev(t) for n, t in v.items()}, {n: _f64(t) for n, t in v.items() if n != "lens"}
    mask = torch.ones(B, dtype=torch.uint8)
    mask[B // 2:] = torch.arange(B - B // 2) % 2 == 0
    lens = [int(m) for m in mask]
    (wo, ws), (bo, bs) = ref.walk(f["q"], f["k"], f["v"], f["log_decay"], lens, f["state"], cfg.scale, dtype)
    keep = d["state"].clone()
    out, state = h.step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], d["state"], mask=mask.cuda(),
                        state_out=torch.empty_like(keep))
    check("out", out, wo[:, 0], bo[:, 0])
    check("state", state, ws, bs)
    assert torch.equal(d["state"], keep) and all(torch.equal(state[b], keep[b]) for b in range(B) if not mask[b])
    out2, state2 = h.step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], d["state"], mask=mask.cuda())
    assert state2 is d["state"] and torch.equal(state2, state) and torch.equal(out2, out)


def test_bits_repeat_and_graphs():
    for L in (130, 1500):
        h, d, want = _case(2, L, 2, 64, 96, "bf16")
        args = [d[n] for n in ("q", "k", "v", "log_decay")]
        run = lambda: (*h.forward(*args, state_in=d["state"]),  # noqa: E731
                       *h.backward(*args, d["dout"], state_in=d["state"], dstate_out=d["dstate"]))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = run()
        keep = d["v"].clone()
        for i in range(3):
            d["v"].copy_(keep * (1 + i))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, run())), (L, i)
            if i == 0:
                assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    cfg = LinearAttentionConfig(2, 64, 32)
    h, v = _handle(cfg), _inputs(2, 9, 2, 64, 32, "bf16", lens=[9, 3])
    d = {n: _dev(t) for n, t in v.items()}
    q, k, x, g, s = (d[n] for n in ("q", "k", "v", "log_decay", "state"))
    for bad in (lambda: h.forward(q[0], k, x, g), lambda: h.forward(q, k[:, :5], x, g), lambda: h.forward(q.float(), k, x, g),
                lambda: h.forward(q, k, x, None), lambda: h.forward(q, k, x, g[:1]), lambda: h.forward(q, k, x, g.cpu()),
                lambda: h.forward(q, k, x, g, lens=d["lens"].long()), lambda: h.forward(q, k, x, g, state_in=s[:, :1]),
                lambda: h.forward(q, k, x, g, state_in=s.transpose(2, 3)), lambda: h.forward(q.cpu(), k, x, g),
                lambda: h.forward(q, k, x, g, out=x[:1].expand(2, 9, 2, 32)), lambda: h.forward(q[:0], k[:0], x[:0], g),
                lambda: h.backward(q, k, x, g, d["dout"][:1]), lambda: h.backward(q, k, x, g, d["dout"], dstate_out=s[:1]),
                lambda: h.step(q[:, 0], k[:, 0], x[:, 0], g, None), lambda: h.step(q[:, 0], k[:, 0], x, g, s),
                lambda: h.forward(torch.empty(2 * 9 * 2 * 64 + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape), k, x, g)):
        with pytest.raises((ValueError, RuntimeError, AttributeError)):
            bad()
