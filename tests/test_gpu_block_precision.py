"""GPU: bf16 attention is as exact as one rounding of its results allows: neither its softmax weights nor their
gradients lose bits on the way, whatever kernel a size takes.

Bounds.  Those of the 64-bit reference without a rounding of the weights: a weight (or its gradient) enters its
product as a sum of two bf16 values, whose second one leaves 2^-8 of the first one's 2^-8: h^2.  delta, formed
from the stored output, is corrected by e = sum_j p_j (dp_j - delta); with computed weights that are off by the
share s of themselves, delta + e differs from sum_j p_j dp_j by s sum p |dp| + s |delta| + sum p edp and the
sum's n u; the correction of dq takes e from a sum of weights that are rounded once, which adds h |e|."""
import numpy as np
import pytest

from scale_gla_layer_amd.config import BlockAttentionConfig
from tests import block_ref as ref
from tests.gpu_cases import say
from tests.test_gpu_block_attention import _check, _host, _i32, _inputs, _op

pytestmark = pytest.mark.gpu

H = ref.HALF["bf16"]


def _forward_bounds(keep):
    w, v, out = keep["w"], keep["v"], keep["out"]
    eo = (keep["share"] + H * H) * (w @ np.abs(v))
    return ref._heads(eo + H * (np.abs(out) + eo))


def _backward_bounds(keep, dout, cfg, val, live):
    w, s, U, G = keep["w"], keep["share"], ref.U, cfg.heads_q // cfg.heads_kv
    do = np.where(live[:, None, :, None], ref._heads(dout), 0)
    B = do.shape[0]
    dp = do @ keep["v"].swapaxes(2, 3)
    edp = (cfg.d_v + 4) * U * (np.abs(do) @ np.abs(keep["v"]).swapaxes(2, 3))
    n = keep["hit"].sum(3, keepdims=True)
    delta = (do * keep["out"]).sum(3, keepdims=True)
    e = (H + (cfg.d_v + 4) * U) * np.abs(do * keep["out"]).sum(3, keepdims=True)  # the stored output's error, at most
    edelta = (w * ((s + n * U) * (np.abs(dp) + np.abs(delta) + e) + edp)).sum(3, keepdims=True) + s * (np.abs(delta) + e)
    ds = w * (dp - delta) * cfg.scale
    # before the correction the gradient of a score holds e as well, whose lower half is rounded
    eds = cfg.scale * w * ((np.abs(dp - delta) + e) * (s + 4 * U + H * H) + edp + edelta)
    eq = (eds + n * U * np.abs(ds) + cfg.scale * w * e * (H + s)) @ np.abs(keep["k"])
    fold = lambda t: t.reshape(B, cfg.heads_kv, G, *t.shape[2:]).sum(2)  # noqa: E731
    rows = np.repeat(fold(keep["hit"].sum(2)[..., None]), G, axis=1)
    ek = fold((eds.swapaxes(2, 3) + rows * U * np.abs(ds).swapaxes(2, 3)) @ np.abs(keep["q"]))
    ev = fold((w * (s + H * H)).swapaxes(2, 3) @ np.abs(do) + rows * U * (w.swapaxes(2, 3) @ np.abs(do)))
    err = {"dq": ref._heads(eq), "dk": ref._heads(ek), "dv": ref._heads(ev)}
    return {x: err[x] + H * (np.abs(val[x]) + err[x]) for x in err}


FEW = [(4, 1, 64, 64, 64, 4, 2, 1),                                        # single queries
       (4, 2, 128, 128, 32, 6, 2, 90), (3, 1, 80, 256, 128, 3, 1, 300),    # dealt to many waves
       (8, 4, 64, 64, 64, 4, 8, 300), (12, 4, 128, 128, 64, 6, 4, 400), (16, 2, 128, 256, 32, 8, 2, 333)]  # three tiles
MANY = [(8, 8, 64, 64, 32, 8, 26, 330), (16, 4, 64, 128, 64, 4, 16, 270), (16, 4, 128, 128, 64, 4, 16, 270),
        (64, 4, 128, 256, 64, 4, 7, 150), (16, 1, 32, 256, 64, 20, 3, 1400)]


def _case(hq, hkv, dk, dv, block, n, B, L):
    cfg = BlockAttentionConfig(hq, hkv, dk, dv, block, n, 1, 2)
    say(f"precision {cfg} B={B} L={L}")
    S = L if L > 1 else 500
    start = [S - L] * B
    op, t = _op(cfg), _inputs(cfg, B, L, S, 70 + L)
    h = {x: _host(y) for x, y in t.items()}
    sel = op.select(t["q"], op.means(t["k"]), _i32(start), S=S)
    want, _, keep = ref.forward(h["q"], h["k"], h["v"], sel.cpu().numpy(), cfg, start)
    return cfg, op, t, h, sel, start, want, keep


@pytest.mark.parametrize("hq,hkv,dk,dv,block,n,B,L", FEW + MANY)
def test_no_bits_are_lost(hq, hkv, dk, dv, block, n, B, L):
    _, op, t, _, sel, start, want, keep = _case(hq, hkv, dk, dv, block, n, B, L)
    out, _ = op.forward(t["q"], t["k"], t["v"], sel, _i32(start))
    _check("out", out, want["out"], _forward_bounds(keep))


@pytest.mark.parametrize("hq,hkv,dk,dv", [(16, 4, 128, 128), (20, 1, 64, 256)])
def test_no_bits_are_lost_in_steps(hq, hkv, dk, dv):
    cfg = BlockAttentionConfig(hq, hkv, dk, dv, 64, 4, 1, 2)
    B, S = 3, 700
    op, t = _op(cfg), _inputs(cfg, B, 1, S, 71)
    pos = np.array([699, 64, 321])
    row = np.arange(B)
    q, kt, vt = t["q"][:, 0].contiguous(), t["k"][row, pos], t["v"][row, pos]
    means = op.means(t["k"])
    sel = op.select(t["q"], means, _i32(pos), S=S)
    out = op.step(q, kt, vt, t["k"], t["v"], means, _i32(pos))
    want, _, keep = ref.forward(_host(q)[:, None], _host(t["k"]), _host(t["v"]), sel.cpu().numpy(), cfg, pos)
    _check("out", out, want["out"][:, 0], _forward_bounds(keep)[:, 0])


@pytest.mark.parametrize("hq,hkv,dk,dv,block,n,B,L", FEW + MANY)
def test_no_bits_are_lost_in_gradients(hq, hkv, dk, dv, block, n, B, L):
    import torch
    cfg, op, t, h, sel, start, want, keep = _case(hq, hkv, dk, dv, block, n, B, L)
    out = torch.from_numpy(want["out"]).to(t["dout"]).contiguous()
    lse = torch.from_numpy(want["lse"]).float().cuda().contiguous()
    got = op.backward(t["q"], t["k"], t["v"], sel, out, lse, t["dout"], _i32(start))
    val, _ = ref.backward(h["q"], h["k"], h["v"], sel.cpu().numpy(), h["dout"], cfg, start)
    bound = _backward_bounds(keep, h["dout"], cfg, val, ref.positions(B, L, t["k"].shape[1], start) >= 0)
    for name, x in zip(("dq", "dk", "dv"), got):
        _check(name, x, val[name], bound[name])
