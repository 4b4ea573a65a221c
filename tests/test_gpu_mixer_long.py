"""GPU: layer norm, linear attention and window attention over more elements than 32 bits count, and tensors whose
positions lie far apart.  The end of a long sequence is held against the 64-bit reference of that part alone: the decay
forgets what was before, and the window ends."""
import pytest
import torch

from scale_gla_layer_amd.config import LayerNormConfig, LinearAttentionConfig, WindowAttentionConfig
from tests import layer_norm_ref, linear_ref, window_ref
from tests.gpu_cases import say
from tests.test_gpu_layer_norm import TYPE, _f64, check
from tests.test_gpu_window_attention import check as check_window

pytestmark = pytest.mark.gpu
CUT, TAIL = 1 << 20, 77 + 600


def _random(*shape, dtype, g):
    return torch.empty(shape, dtype=TYPE[dtype], device="cuda").normal_(generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm(dtype):
    from scale_gla_layer_amd.runner import DeviceLayerNorm
    D, L, g = 2304, CUT + TAIL, torch.Generator(device="cuda").manual_seed(1)
    say(f"layer norm, long, {dtype}")
    x, dy = (_random(1, L, D, dtype=dtype, g=g) for _ in range(2))
    w, b = (torch.randn(D, generator=g, device="cuda") for _ in range(2))
    dy[:, :CUT] = 0
    op = DeviceLayerNorm(LayerNormConfig(D, dtype=dtype))
    y, mean, rstd = op.forward(x, w, b)
    tail = x[:, CUT:]
    want, bound = layer_norm_ref.forward(_f64(tail), _f64(w), _f64(b), 1e-5, dtype)
    for n, t in (("y", y), ("mean", mean), ("rstd", rstd)):
        check(n, t[:, CUT:], want[n], bound[n])
    dx, dw, db = op.backward(x, dy, mean, rstd, w, b, dx=y)
    want, bound = layer_norm_ref.backward(_f64(tail), _f64(dy[:, CUT:]), _f64(mean[:, CUT:]), _f64(rstd[:, CUT:]), _f64(w), dtype)
    for n, t in (("dx", dx[:, CUT:]), ("dweight", dw), ("dbias", db)):  # rows without a gradient add 0
        check(n, t, want[n], bound[n])
    assert not dx[:, :CUT].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_attention(dtype):
    from scale_gla_layer_amd.runner import DeviceLinearAttention
    H, dk, dv, L, g = 16, 128, 144, CUT + TAIL, torch.Generator(device="cuda").manual_seed(2)
    say(f"linear attention, long, {dtype}")
    q, k = (_random(1, L, H, dk, dtype=dtype, g=g) for _ in range(2))
    v, do = (_random(1, L, H, dv, dtype=dtype, g=g) for _ in range(2))
    ld = torch.full((H,), -1.5, device="cuda")  # e^-150 of the state is left after 100 positions
    op = DeviceLinearAttention(LinearAttentionConfig(H, dk, dv, dtype=dtype))
    out, last = op.forward(q, k, v, ld)
    part = 260
    f = [_f64(t[:, -part:]) for t in (q, k, v)]
    (wo, ws), (bo, bs) = linear_ref.walk(*f, _f64(ld), [part], None, dk ** -0.5, dtype)
    check("out", out[:, -150:], wo[:, -150:], bo[:, -150:])
    check("state", last, ws, bs)
    dq, dk_, dv_, _ = op.backward(q, k, v, ld, do)
    want, bound = linear_ref.backward(*f, _f64(ld), [part], None, _f64(do[:, -part:]), None, dk ** -0.5, dtype)
    for n, t in (("dq", dq), ("dk", dk_), ("dv", dv_)):
        check(n, t[:, -150:], want[n][:, -150:], bound[n][:, -150:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention(dtype):
    from scale_gla_layer_amd.runner import DeviceWindowAttention
    H, d, L, g, part, sink = 17, 128, CUT + TAIL, torch.Generator(device="cuda").manual_seed(3), 400, 4
    cfg = WindowAttentionConfig(H, H, d, d, 90, sink, None, dtype)
    say(f"window attention, long, {dtype}")
    op = DeviceWindowAttention(cfg)
    q, k, v, do = (_random(1, L, H, d, dtype=dtype, g=g) for _ in range(4))

    def tail(t, n=part):  # the first tokens and the last n positions
        return torch.cat([t[:, :sink], t[:, -n:]], 1).double()

    gathered = q[:, -part:].double(), tail(k), tail(v)
    want, bound, _ = window_ref.forward(*gathered, cfg, [sink])
    out, lse = op.forward(q, k, v)
    check_window("out", out[:, -200:], want["out"][:, -200:], bound["out"][:, -200:])
    check_window("lse", lse[:, :, -200:], want["lse"][:, :, -200:], bound["lse"][:, :, -200:])
    # a few rows of the same
    some, some_lse = op.forward(q[:, -30:].contiguous(), k, v, start=torch.tensor([L - 30], dtype=torch.int32, device="cuda"))
    check_window("few rows", some, want["out"][:, -30:], bound["out"][:, -30:])
    dq, dk, dv = op.backward(q, k, v, out, lse, do)
    wg, bg = window_ref.backward(*gathered, do[:, -part:].double(), cfg, [sink])
    check_window("dq", dq[:, -200:], wg["dq"][:, -200:], bg["dq"][:, -200:])
    for n, t in (("dk", dk), ("dv", dv)):
        check_window(n, t[:, -200:], wg[n][:, -200:], bg[n][:, -200:])
    # a step at the end of the cache, and an append there
    one = [t[:, 0].contiguous() for t in (q, k, v)]
    pos = torch.tensor([L - 1], dtype=torch.int32, device="cuda")
    ot = op.step(*one, k, v, pos)
    assert torch.equal(k[:, -1], one[1]) and torch.equal(v[:, -1], one[2])
    want, bound, _ = window_ref.forward(one[0][:, None].double(), tail(k), tail(v), cfg, [sink + part - 1])
    check_window("step", ot[:, None], want["out"], bound["out"])
    fresh = (k[:, 5:25].contiguous(), v[:, 5:25].contiguous())
    before = k[:, -21].clone()
    op.append(*fresh, k, v, pos=pos - 19)
    assert torch.equal(k[:, -20:], fresh[0]) and torch.equal(v[:, -20:], fresh[1]) and torch.equal(k[:, -21], before)


def test_positions_far_apart():
    """Views whose positions lie 160 MB apart: offsets within one tile pass 32 bits."""
    from scale_gla_layer_amd.runner import DeviceLayerNorm, DeviceLinearAttention, DeviceWindowAttention
    L, H, d, far = 70, 2, 64, 80 << 20
    say("positions far apart")
    g = torch.Generator(device="cuda").manual_seed(4)
    room = torch.zeros(L * far, dtype=torch.bfloat16, device="cuda")
    n = [0]

    def view(t):
        out = room[n[0]:].as_strided((1, L, *t.shape[2:]), (0, far, *t.stride()[2:]))
        n[0] += t[0, 0].numel() + 64
        return out.copy_(t)

    q, k, v, do = (_random(1, L, H, d, dtype="bf16", g=g) for _ in range(4))
    far_q, far_k, far_v, far_do = (view(t) for t in (q, k, v, do))
    lin, ld = DeviceLinearAttention(LinearAttentionConfig(H, d, d)), torch.tensor([-0.1, -0.01], device="cuda")
    a, b = lin.forward(q, k, v, ld), lin.forward(far_q, far_k, far_v, ld, out=view(torch.zeros_like(v)))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = lin.backward(q, k, v, ld, do), lin.backward(far_q, far_k, far_v, ld, far_do, dq=view(q), dk=view(k), dv=view(v))
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    for win in (DeviceWindowAttention(WindowAttentionConfig(H, H, d, d, 40, 3)), DeviceWindowAttention(WindowAttentionConfig(H, 1, d, d, 40, 3))):
        kk, vv, fk, fv = (t[:, :, :win.cfg.heads_kv] for t in (k, v, far_k, far_v))
        kk, vv = kk.contiguous(), vv.contiguous()
        (out, lse), (fo, flse) = win.forward(q, kk, vv), win.forward(far_q, fk, fv, out=view(torch.zeros_like(q)))
        assert torch.equal(out, fo) and torch.equal(lse, flse)
        a = win.backward(q, kk, vv, out, lse, do)
        b = win.backward(far_q, fk, fv, fo, lse, far_do, dq=view(q), dk=view(kk), dv=view(vv))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    norm = DeviceLayerNorm(LayerNormConfig(H * d))
    x, fx, y = (t.flatten(2) for t in (q, far_q, do))
    a, b = norm.forward(x), norm.forward(fx)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert torch.equal(norm.backward(x, y, *a[1:])[0], norm.backward(fx, far_do.flatten(2), *a[1:])[0])
