"""CPU: the 64-bit block attention's gradients against central differences, its
selection against a hand-made case, and the refusals of the C entry points, the
configuration and the device handle."""
import ctypes

import numpy as np
import pytest

from scale_gla_layer_amd import binding
from scale_gla_layer_amd.config import BlockAttentionConfig
from tests import block_ref as ref


def test_gradients_against_differences():
    rng = np.random.default_rng(2)
    cfg = BlockAttentionConfig(4, 2, 8, 8, 32, 2, 1, 1, dtype="f32")
    B, L = 1, 70
    t = {"q": rng.normal(size=(B, L, 4, 8)), "k": rng.normal(size=(B, L, 2, 8)), "v": rng.normal(size=(B, L, 2, 8))}
    dout = rng.normal(size=(B, L, 4, 8))
    sel = ref.select(t["q"], ref.means(t["k"], 32), cfg, L)
    lens = np.array([66])
    g = ref.backward(t["q"], t["k"], t["v"], sel, dout, cfg, lens=lens)[0]

    def loss(**kw):
        a = {**t, **kw}
        return (ref.forward(a["q"], a["k"], a["v"], sel, cfg, lens=lens)[0]["out"] * dout).sum()

    for name in t:
        for at in [tuple(rng.integers(0, n) for n in t[name].shape) for _ in range(25)]:
            up, down = t[name].copy(), t[name].copy()
            up[at] += 1e-5
            down[at] -= 1e-5
            assert abs((loss(**{name: up}) - loss(**{name: down})) / 2e-5 - g["d" + name][at]) < 1e-8


def test_selection_by_hand():
    cfg = BlockAttentionConfig(1, 1, 8, 8, 32, 4, 1, 1, dtype="f32")
    c = np.zeros((1, 1, 8, 8))
    c[0, 0, :, 0] = [0, 3, 1, 3, -1, 2, 9, 9]
    q = np.zeros((1, 3, 1, 8))
    q[..., 0] = 1
    got = ref.select(q, c, cfg, 256, start=np.array([6 * 32 - 1]))[0, 0]  # positions 191, 192, 193
    assert got.tolist() == [[0, 1, 3, 5], [0, 1, 3, 6], [0, 1, 3, 6]]
    assert ref.select(-q, c, cfg, 256, start=np.array([255]))[0, 0].tolist()[0] == [0, 2, 4, 7]
    assert ref.select(q, c, cfg, 256, lens=np.array([1]))[0, 0].tolist() == [[0, -1, -1, -1], [-1] * 4, [-1] * 4]


GOOD = dict(heads_q=8, heads_kv=2, d_k=64, d_v=64, block=64, n_select=8, n_first=1, n_recent=2, scale=0.125, dtype=1)


def _raw(**kw):
    c = {**GOOD, **kw}
    return ctypes.byref(binding.CBlockConfig(*(c[n] for n in GOOD)))


BAD_SIZE = 2 ** 64 - 1


@pytest.mark.parametrize("bad", [
    dict(heads_kv=0), dict(heads_q=7), dict(heads_q=1), dict(heads_q=1026), dict(d_k=4), dict(d_k=136), dict(d_k=60),
    dict(d_v=0), dict(d_v=264), dict(block=16), dict(block=96), dict(n_select=0), dict(n_select=65), dict(n_first=-1),
    dict(n_recent=0), dict(n_first=7), dict(n_first=2 ** 31 - 1, n_recent=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=0.0), dict(scale=-0.1), dict(dtype=2)])
def test_invalid_configurations(bad):
    lib, c = binding.load_library(), _raw(**bad)
    assert lib.msgla_block_attention_workspace_bytes(c, 1, 8, 8) == BAD_SIZE
    assert lib.msgla_block_attention_backward_workspace_bytes(c, 1, 8, 8) == BAD_SIZE
    assert lib.msgla_block_attention_step_workspace_bytes(c, 1, 8) == BAD_SIZE
    t = ctypes.byref(binding.CHeads(4096, 1024, 64, 64))
    assert lib.msgla_block_means(c, t, None, None, 1, 8, 4096, None) == 1
    assert lib.msgla_block_select(c, t, 4096, None, None, 1, 8, 8, 4096, None) == 1
    if all(n in BlockAttentionConfig.__dataclass_fields__ for n in bad) and "dtype" not in bad:
        with pytest.raises(ValueError):
            BlockAttentionConfig(**{**GOOD, "dtype": "bf16", **bad})


@pytest.mark.parametrize("B,L,S", [(0, 1, 8), (1, 0, 8), (1, 8, 0), (1, 8, (1 << 24) + 1), (1 << 12, 1 << 17, 8)])
def test_invalid_sizes(B, L, S):
    lib = binding.load_library()
    assert lib.msgla_block_attention_workspace_bytes(_raw(), B, L, S) == BAD_SIZE
    assert lib.msgla_block_attention_backward_workspace_bytes(_raw(), B, L, S) == BAD_SIZE
    t = ctypes.byref(binding.CHeads(4096, 1024, 64, 64))
    assert lib.msgla_block_attention(_raw(), t, t, t, 4096, None, None, B, L, S, t, None, 4096, 1 << 62, None) == 1


def test_bad_arguments_return_before_anything_is_enqueued():
    lib, c = binding.load_library(), _raw()
    t = lambda p=4096, b=1024, s=64, h=64: ctypes.byref(binding.CHeads(p, b, s, h))  # noqa: E731
    ok = t()
    assert lib.msgla_block_means(c, None, None, None, 1, 8, 4096, None) == 1
    for bad in (t(0), t(4104), t(b=-8), t(s=12), t(h=4)):
        assert lib.msgla_block_means(c, bad, None, None, 1, 8, 4096, None) == 1
        assert lib.msgla_block_select(c, bad, 4096, None, None, 1, 8, 8, 4096, None) == 1
    assert lib.msgla_block_means(c, ok, 4098, None, 1, 8, 4096, None) == 1
    assert lib.msgla_block_means(c, ok, None, None, 1, 8, None, None) == 1
    assert lib.msgla_block_select(c, ok, 4096, None, None, 1, 8, 8, None, None) == 1
    need = lib.msgla_block_attention_workspace_bytes(c, 1, 8, 8)
    assert 0 < need < BAD_SIZE
    fwd = lambda q=ok, sel=4096, ws=4096, n=need, out=ok: lib.msgla_block_attention(  # noqa: E731
        c, q, ok, ok, sel, None, None, 1, 8, 8, out, None, ws, n, None)
    assert fwd(q=None) == 1 and fwd(sel=None) == 1 and fwd(ws=None) == 1 and fwd(ws=4100) == 1 and fwd(out=t(0)) == 1
    assert fwd(n=need - 1) == 3
    need = lib.msgla_block_attention_backward_workspace_bytes(c, 1, 8, 8)
    bwd = lambda lse=4096, dq=ok, n=need: lib.msgla_block_attention_backward(  # noqa: E731
        c, ok, ok, ok, 4096, None, None, ok, lse, ok, 1, 8, 8, dq, ok, ok, 4096, n, None)
    assert bwd(lse=None) == 1 and bwd(dq=None) == 1 and bwd(n=need - 1) == 3
    need = lib.msgla_block_attention_step_workspace_bytes(c, 1, 8)
    step = lambda pos=4096, m=4096, n=need: lib.msgla_block_attention_step(  # noqa: E731
        c, ok, ok, ok, pos, 1, 8, ok, ok, m, ok, 4096, n, None)
    assert step(pos=None) == 1 and step(m=None) == 1 and step(n=need - 1) == 3


def test_handle_refuses_host_tensors():
    import torch
    from scale_gla_layer_amd.runner import DeviceBlockAttention
    op = DeviceBlockAttention(BlockAttentionConfig(8, 2, 64, 64))
    with pytest.raises(ValueError, match="ROCm device"):
        op.means(torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="must be given"):
        op.means(torch.zeros(1, 8, 2, 64), start_from=torch.zeros(1, dtype=torch.int32))
