"""GPU: block selection and attention at the ends of what their launches and documents allow."""
import numpy as np
import pytest

from scale_gla_layer_amd.config import BlockAttentionConfig
from tests import block_ref as ref
from tests.test_gpu_block_attention import _check, _host, _i32, _inputs, _op
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


@pytest.mark.parametrize("dtype,d,grad", [("bf16", 64, False), ("bf16", 128, True), ("f32", 128, False)])
def test_the_longest_lists_of_the_largest_workgroups(dtype, d, grad):
    """A head of queries for each of keys, 64 of 256 blocks chosen, 4096 tiles: maps and lists leave the ring
    of key stages not a byte more than the compute unit has."""
    torch = _torch()
    H, L, T, n = 4, 16384, 64, 64
    cfg = BlockAttentionConfig(H, H, d, d, T, n, 1, 2, None, dtype)
    say(f"longest lists {dtype} {d}")
    op, t = _op(cfg), _inputs(cfg, 1, L, L, 41)
    sel = op.select(t["q"], op.means(t["k"]))
    out, lse = op.forward(t["q"], t["k"], t["v"], sel)
    rows = np.array([0, T - 1, 4097, 9000, L - T, L - 1])  # each as a sequence of one query
    q, do = (_host(t[x])[0, rows][:, None] for x in ("q", "dout"))
    k, v = (np.repeat(_host(t[x]), len(rows), axis=0) for x in "kv")
    chosen = np.moveaxis(sel.cpu().numpy()[0][:, rows], 1, 0)[:, :, None]
    want, bound, _ = ref.forward(q, k, v, chosen, cfg, rows)
    _check("out", out[0, rows][:, None], want["out"], bound["out"])
    _check("lse", lse[0][:, rows].t()[:, :, None], want["lse"], bound["lse"])
    if grad:
        dq, dk, dv = op.backward(t["q"], t["k"], t["v"], sel, out, lse, t["dout"])
        want, bound = ref.backward(q, k, v, chosen, do, cfg, rows)
        _check("dq", dq[0, rows][:, None], want["dq"], bound["dq"])
        assert bool(dk.isfinite().all()) and bool(dv.isfinite().all())


def test_a_chunk_that_runs_past_the_cache():
    """Rows behind a cache whose last block is not whole select nothing, as the attention leaves them out."""
    cfg = BlockAttentionConfig(8, 2, 64, 64, 64, 4)
    B, L, S, start = 3, 40, 700, [690, 660, 699]
    op, t = _op(cfg), _inputs(cfg, B, L, S, 42)
    means = op.means(t["k"])
    sel = op.select(t["q"], means, _i32(start), S=S)
    assert np.array_equal(sel.cpu().numpy(), ref.select(_host(t["q"]), _host(means), cfg, S, start))
    out, lse = op.forward(t["q"], t["k"], t["v"], sel, _i32(start))
    behind = _torch().tensor(ref.positions(B, L, S, start) < 0).cuda()
    assert behind.sum() == 30 + 39 and bool((sel.transpose(1, 2)[behind] == -1).all())
    assert bool((out[behind] == 0).all()) and bool((lse.transpose(1, 2)[behind] == -float("inf")).all())
    with pytest.raises(ValueError):
        op.select(t["q"], means, _i32(start), S=S + 64)


def test_gradients_of_many_short_sequences():
    """More sequences and key-value heads than a grid's second dimension would count."""
    torch = _torch()
    cfg = BlockAttentionConfig(2, 2, 8, 16, 32, 1, 0, 1)
    B, L = 40000, 2
    op, t = _op(cfg), _inputs(cfg, B, L, L, 43)
    sel = torch.zeros((B, 2, L, 1), dtype=torch.int32, device="cuda")
    out, lse = op.forward(t["q"], t["k"], t["v"], sel)
    h = {n: _host(x) for n, x in t.items()}
    want, bound, _ = ref.forward(h["q"], h["k"], h["v"], sel.cpu().numpy(), cfg)
    _check("out", out, want["out"], bound["out"])
    out, lse = torch.from_numpy(want["out"]).to(out).contiguous(), torch.from_numpy(want["lse"]).to(lse).contiguous()
    got = op.backward(t["q"], t["k"], t["v"], sel, out, lse, t["dout"])
    want, bound = ref.backward(h["q"], h["k"], h["v"], sel.cpu().numpy(), h["dout"], cfg)
    for name, x in zip(("dq", "dk", "dv"), got):
        _check(name, x, want[name], bound[name])


def test_caches_beyond_32_bits():
    """The last of five sequences whose caches hold 5 GB each, against that sequence alone."""
    torch = _torch()
    cfg = BlockAttentionConfig(16, 8, 64, 64, 64, 16)
    B, S = 5, 1 << 20
    op = _op(cfg)
    g = torch.Generator(device="cuda").manual_seed(44)
    k, v = (torch.empty((B, S, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (*k, *v):
        x.normal_(generator=g)
    q, kt, vt = (torch.randn((B, n, 64), generator=g, device="cuda").bfloat16() for n in (16, 8, 8))
    pos = _i32([5, S - 1, 77, S // 2 + 63, S - 1])
    last, k1, v1 = slice(B - 1, B), k[B - 1:].clone(), v[B - 1:].clone()
    means = op.means(k, pos)
    assert torch.equal(means[last], op.means(k1, pos[last]))
    sel = op.select(q[:, None], means, pos)
    assert torch.equal(sel[last], op.select(q[last, None], means[last].contiguous(), pos[last]))
    for a, b in zip(op.forward(q[:, None], k, v, sel, pos), op.forward(q[last, None], k1, v1, sel[last], pos[last])):
        assert torch.equal(a[last], b)
    m1 = means[last].clone()
    out = op.step(q, kt, vt, k, v, means, pos)
    assert torch.equal(out[last], op.step(q[last], kt[last], vt[last], k1, v1, m1, pos[last]))
    assert torch.equal(k[last], k1) and torch.equal(v[last], v1) and torch.equal(means[last], m1)
