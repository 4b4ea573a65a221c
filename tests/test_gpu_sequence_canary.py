"""GPU: every buffer that the sequence operators write (outputs, states, caches, workspaces of exactly the
queried size) with a guard band on both sides: no guard byte changes, and the results are those of
unguarded buffers bit for bit.  Workspaces in the wrong place are refused."""
import numpy as np
import pytest

from scale_gla_layer_amd import binding
from scale_gla_layer_amd.config import BlockAttentionConfig, RecurrenceConfig
from tests.gpu_cases import say
from tests.test_gpu_block_attention import _i32
from tests.test_gpu_block_attention import _inputs as block_inputs
from tests.test_gpu_canary import Guarded
from tests.test_gpu_recurrence import _inputs as recurrence_inputs

pytestmark = pytest.mark.gpu


class Buffers:
    """Buffers for outputs, guarded or not."""

    def __init__(self, guarded):
        self.guarded, self.all = guarded, []

    def __call__(self, shape, dtype, fill=0x5A):
        import torch
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        if not self.guarded:
            # other contents: what the calls leave may not depend on what they found
            return torch.full((n,), 0xFF - fill, dtype=torch.uint8, device="cuda").view(dtype).view(shape)
        self.all.append(Guarded(n, fill))
        return self.all[-1].body.view(dtype).view(shape)

    def like(self, t):
        return self(tuple(t.shape), t.dtype)

    def copy(self, t):
        return self.like(t).copy_(t)

    def room(self, n):
        import torch
        return self((n,), torch.uint8, 0xA5)


def _both(run):
    import torch
    plain, bufs = run(Buffers(False)), Buffers(True)
    got = run(bufs)
    torch.cuda.synchronize()
    assert bufs.all and all(b.intact() for b in bufs.all)
    for i, (a, b) in enumerate(zip(got, plain)):
        assert torch.equal(a.nan_to_num(), b.nan_to_num()), f"output {i}"


@pytest.mark.parametrize("B,L,D,dtype,mode,mask", [
    (3, 40, 7, "f32", "convex", "holes"), (2, 100, 64, "bf16", "norm", None), (2, 3000, 130, "bf16", "plain", "ragged"),
    (1, 2100, 65, "f32", "norm", None)])
def test_recurrence(B, L, D, dtype, mode, mask):
    import torch
    say(f"canary recurrence B={B} L={L} D={D} {dtype} {mode} {mask}")
    cfg = RecurrenceConfig(D, mode, 16.0, dtype)
    d = {n: None if t is None else t.cuda() for n, t in recurrence_inputs(B, L, D, dtype, 60, mask).items()}
    step_mask = None if d["mask"] is None else d["mask"][:, 0].contiguous()

    def run(buf):
        y, h = buf.like(d["x"]), buf.like(d["h_in"])
        binding.msgla_recurrence_forward(cfg, d["x"], d["z"], y, buf.room(binding.msgla_recurrence_workspace_bytes(cfg, B, L)),
                                         d["bias"], d["mask"], d["h_in"], h)
        dx, dz, db, dh = (buf.like(d[n]) for n in ("x", "z", "bias", "h_in"))
        binding.msgla_recurrence_backward(cfg, d["x"], d["z"], d["dy"], dx, dz,
                                          buf.room(binding.msgla_recurrence_backward_workspace_bytes(cfg, B, L)), d["bias"],
                                          d["mask"], d["h_in"], d["dh_out"], db, dh)
        yt, ht = buf((B, D), d["x"].dtype), buf.like(d["h_in"])
        binding.msgla_recurrence_step(cfg, d["x"][:, 0], d["z"][:, 0], yt, d["h_in"], ht, d["bias"], step_mask)
        return [y, h, dx, dz, db, dh, yt, ht]

    _both(run)
    with pytest.raises(ValueError, match="workspace"):
        binding.msgla_recurrence_forward(cfg, d["x"], d["z"], torch.empty_like(d["x"]), torch.empty(1 << 22, dtype=torch.uint8))


@pytest.mark.parametrize("hq,hkv,dk,dv,block,n,B,L,S,dtype", [
    (4, 2, 64, 64, 32, 4, 2, 5, 90, "bf16"),          # few queries, dealt to many waves
    (6, 2, 80, 96, 32, 6, 3, 333, 401, "f32"),        # workgroups of three tiles
    (20, 1, 64, 256, 128, 3, 2, 130, 300, "bf16"),    # two tiles a query
    (8, 8, 64, 64, 32, 4, 26, 330, 330, "bf16"),      # workgroups of fifteen
    (64, 4, 128, 256, 64, 4, 7, 150, 200, "bf16"),    # of eleven
    (4, 1, 128, 128, 64, 40, 1, 1000, 8333, "bf16"),  # a block's queries in several work items; a long cache
])
def test_blocks(hq, hkv, dk, dv, block, n, B, L, S, dtype):
    import torch
    cfg = BlockAttentionConfig(hq, hkv, dk, dv, block, n, 1, 2, None, dtype)
    say(f"canary {cfg} B={B} L={L} S={S}")
    t = block_inputs(cfg, B, L, S, 61)
    rng = np.random.default_rng(62)
    start = rng.integers(0, S - L + 1, B)
    start[0] = S - L
    lens = _i32(np.minimum(start + rng.integers(1, L + 1, B), S))
    pos, start = _i32(rng.integers(0, S, B)), _i32(start)
    nb = binding.block_count(cfg, S)
    f32 = torch.float32

    def run(buf):
        means, sel = buf((B, hkv, nb, dk), f32), buf((B, hkv, L, n), torch.int32)
        binding.msgla_block_means(cfg, t["k"], means, lens)
        binding.msgla_block_select(cfg, t["q"], means, S, sel, start, lens)
        out, lse = buf((B, L, hq, dv), t["q"].dtype), buf((B, hq, L), f32)
        room = buf.room(binding.msgla_block_attention_workspace_bytes(cfg, B, L, S))
        binding.msgla_block_attention(cfg, t["q"], t["k"], t["v"], sel, out, lse, room, start, lens)
        g = [buf.like(t[x]) for x in "qkv"]
        room = buf.room(binding.msgla_block_attention_backward_workspace_bytes(cfg, B, L, S))
        binding.msgla_block_attention_backward(cfg, t["q"], t["k"], t["v"], sel, out, lse, t["dout"], *g, room, start, lens)
        k, v, m, o = buf.copy(t["k"]), buf.copy(t["v"]), buf.copy(means), buf((B, hq, dv), t["q"].dtype)
        room = buf.room(binding.msgla_block_attention_step_workspace_bytes(cfg, B, S))
        binding.msgla_block_attention_step(cfg, t["q"][:, 0], t["k"][:, 1], t["v"][:, 1], k, v, m, pos, o, room)
        return [means, sel, out, lse, *g, k, v, m, o]

    _both(run)
    sel = torch.zeros((B, hkv, L, n), dtype=torch.int32, device="cuda")
    for room in (torch.empty(1 << 28, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 28)):
        with pytest.raises(ValueError, match="workspace"):
            binding.msgla_block_attention(cfg, t["q"], t["k"], t["v"], sel, torch.zeros_like(t["dout"]), None, room)
