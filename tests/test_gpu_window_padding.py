"""GPU: window attention where a position that is used holds a NaN or an infinity: outputs of padding stay 0, their
logarithm minus infinity and their gradients 0, in tiles shared with rows that the NaN reaches; other sequences keep
their bits."""
import pytest
import torch

from scale_gla_layer_amd.config import WindowAttentionConfig
from tests.gpu_cases import say
from tests.test_gpu_layer_norm import TYPE
from tests.test_gpu_window_attention import _handle, _i32, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["q", "k", "v", "do"])
@pytest.mark.parametrize("B,L,hq,hkv,dk,dv,window,n_sink,lens,start", [
    (2, 9, 8, 2, 64, 64, 100, 4, [2, 9], None),            # a few rows, padding in the tile of the NaN's rows
    (2, 9, 3, 1, 64, 256, 4, 0, [3, 9], None),
    (1, 40, 1, 1, 32, 64, 7, 3, [21], [-5]),               # padding before the sequence as well
    (3, 30, 4, 1, 128, 128, 4000, 2, [25, 1, 30], None),
    (70, 120, 2, 2, 64, 128, 50, 40, [120, 37] + [110] * 68, None),  # many rows
    (6, 1100, 4, 2, 64, 96, 300, 4, [1100, 1099, 3, 0, 513, 700], None),  # first tokens behind the window
])
def test_padding_beside_a_nan(B, L, hq, hkv, dk, dv, window, n_sink, lens, start, what, dtype):
    say(f"padding beside a NaN B={B} L={L} heads={hq}/{hkv} d={dk}/{dv} window={window} sinks={n_sink} {what} {dtype}")
    cfg = WindowAttentionConfig(hq, hkv, dk, dv, window, n_sink, None, dtype)
    h, (q, k, v, do) = _handle(cfg), _inputs(B, L, L, cfg, 2)
    s, n = _i32(start), _i32(lens)
    clean = h.forward(q, k, v, start=s, lens=n)
    clean = (*clean, *h.backward(q, k, v, *clean, do, start=s, lens=n))
    first = 0 if start is None else -start[0]  # the first row that is no padding
    {"q": q, "k": k, "v": v, "do": do}[what][0, first if what in ("q", "do") else 0, 0, 1] = float("nan" if dtype == "bf16" else "inf")
    out, lse = h.forward(q, k, v, start=s, lens=n)
    dq, dk_, dv_ = h.backward(q, k, v, out, lse, do, start=s, lens=n)
    at = torch.arange(L, device="cuda")
    for b in range(B):
        p = at + (0 if start is None else start[b])
        pad = (p < 0) | (p >= lens[b])
        assert (out[b, pad] == 0).all() and (lse[b, :, pad] == -float("inf")).all() and (dq[b, pad] == 0).all(), b
        if b:
            assert all(torch.equal(x[b], y[b]) for x, y in zip(clean, (out, lse, dq, dk_, dv_))), b
    assert not all(torch.isfinite(t[0]).all() for t in (out, dq, dk_, dv_))  # it is used


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_without_a_place_beside_a_nan(dtype):
    cfg = WindowAttentionConfig(4, 2, 64, 96, 1000, 2, None, dtype)
    h, (q, k, v, _) = _handle(cfg), _inputs(3, 1, 1100, cfg, 4)
    qt, kt, vt = (t[:, 0].contiguous() for t in _inputs(3, 1, 1, cfg, 5)[:3])
    k[1], v[1], kt[1], vt[1] = (torch.full((), float("nan"), dtype=TYPE[dtype], device="cuda") for _ in range(4))
    pos = _i32([500, -1, 5000])
    out = h.step(qt, kt, vt, k, v, pos)
    assert (out[1] == 0).all() and torch.isfinite(out[::2].float()).all() and k[1].isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_that_sits_out(dtype):
    """pos below 0: append and step leave the sequence's cache as it is, also where tokens would reach positions from 0 on."""
    cfg = WindowAttentionConfig(4, 2, 64, 64, 20, 3, None, dtype)
    h, (_, k, v, _), (q, kn, vn, _) = _handle(cfg), _inputs(4, 1, 30, cfg, 6), _inputs(4, 50, 50, cfg, 7)
    pos = _i32([0, -1, -7, 12])
    want_k, want_v = k.clone(), v.clone()
    h.append(kn, vn, k, v, pos=pos)
    out = h.step(q[:, 0], kn[:, 3], vn[:, 3], k, v, pos)
    for b in (1, 2):
        assert torch.equal(k[b], want_k[b]) and torch.equal(v[b], want_v[b]) and (out[b] == 0).all()
    for b in (0, 3):
        assert not torch.equal(k[b], want_k[b]) and (out[b] != 0).any()
