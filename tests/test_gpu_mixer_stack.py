"""GPU: layer norm, linear attention and window attention together, as a model uses them: x + linear(norm(x)), then
x + window(norm(x)), over a padded batch.  A prompt's pass, single tokens after it from the state and the rolling cache
that it left, and the gradient of the whole, each call held against the 64-bit reference of what it was given; two
streams at once; and the whole captured and replayed."""
import pytest
import torch

from scale_gla_layer_amd.config import LayerNormConfig, LinearAttentionConfig, WindowAttentionConfig
from tests import layer_norm_ref, linear_ref, window_ref
from tests.gpu_cases import say
from tests.test_gpu_layer_norm import TYPE, _f64, check
from tests.test_gpu_window_attention import _i32
from tests.test_gpu_window_attention import check as check_window

pytestmark = pytest.mark.gpu
B, H, HKV, D, EPS = 3, 4, 2, 64, 1e-5
WIDTH = H * D


class Stack:
    """Two mixers.  Projections are fixed matrices of the storage type, plain products of torch."""

    def __init__(self, dtype, window=50, n_sink=3):
        from scale_gla_layer_amd.runner import DeviceLayerNorm, DeviceLinearAttention, DeviceWindowAttention
        g = torch.Generator().manual_seed(9)
        self.dtype, self.T = dtype, TYPE[dtype]
        self.norm = DeviceLayerNorm(LayerNormConfig(WIDTH, EPS, dtype))
        self.lin = DeviceLinearAttention(LinearAttentionConfig(H, D, D, dtype=dtype))
        self.win = DeviceWindowAttention(WindowAttentionConfig(H, HKV, D, D, window, n_sink, None, dtype))
        r = lambda *n: torch.randn(n, generator=g)  # noqa: E731
        self.w1, self.w2 = ((r(WIDTH, n * D) * WIDTH ** -0.5).to(self.T).cuda() for n in (3 * H, H + 2 * HKV))
        self.nw, self.nb = [(1 + 0.2 * r(WIDTH)).cuda() for _ in range(2)], [(0.2 * r(WIDTH)).cuda() for _ in range(2)]
        self.ld = torch.tensor([-0.3, -0.05, -0.01, 0.0], device="cuda")

    def split(self, y, w, *heads):
        parts = (y @ w).split([n * D for n in heads], -1)
        return [p.unflatten(-1, (n, D)) for p, n in zip(parts, heads)]

    def forward(self, x, lens=None, state=None):
        """What every call was given and what it gave."""
        f = {"x0": x}
        f["y0"], f["mean0"], f["rstd0"] = self.norm.forward(x, self.nw[0], self.nb[0])
        f["q0"], f["k0"], f["v0"] = self.split(f["y0"], self.w1, H, H, H)
        f["o0"], f["state"] = self.lin.forward(f["q0"], f["k0"], f["v0"], self.ld, lens=lens, state_in=state)
        f["x1"] = x + f["o0"].flatten(2)
        f["y1"], f["mean1"], f["rstd1"] = self.norm.forward(f["x1"], self.nw[1], self.nb[1])
        f["q1"], f["k1"], f["v1"] = self.split(f["y1"], self.w2, H, HKV, HKV)
        f["o1"], f["lse"] = self.win.forward(f["q1"], f["k1"], f["v1"], lens=lens)
        f["x2"] = f["x1"] + f["o1"].flatten(2)
        return f

    def backward(self, f, dx2, lens=None):
        """The gradient of x0 and of the norms' parameters; b: what every call was given and gave."""
        b = {"do1": dx2.unflatten(2, (H, D))}
        b["dq1"], b["dk1"], b["dv1"] = self.win.backward(f["q1"], f["k1"], f["v1"], f["o1"], f["lse"], b["do1"], lens=lens)
        b["dy1"] = torch.cat([b[n].flatten(2) for n in ("dq1", "dk1", "dv1")], -1) @ self.w2.T
        b["dn1"], b["dw1"], b["db1"] = self.norm.backward(f["x1"], b["dy1"], f["mean1"], f["rstd1"], self.nw[1], self.nb[1])
        b["dx1"] = dx2 + b["dn1"]
        b["do0"] = b["dx1"].unflatten(2, (H, D))
        b["dq0"], b["dk0"], b["dv0"], _ = self.lin.backward(f["q0"], f["k0"], f["v0"], self.ld, b["do0"], lens=lens)
        b["dy0"] = torch.cat([b[n].flatten(2) for n in ("dq0", "dk0", "dv0")], -1) @ self.w1.T
        b["dn0"], b["dw0"], b["db0"] = self.norm.backward(f["x0"], b["dy0"], f["mean0"], f["rstd0"], self.nw[0], self.nb[0])
        b["dx0"] = b["dx1"] + b["dn0"]
        return b

    def step(self, x, state, k, v, pos):
        """One token x [B, WIDTH] of every sequence; the state and the caches are renewed."""
        f = {"x0": x[:, None]}
        f["y0"], *_ = self.norm.forward(f["x0"], self.nw[0], self.nb[0])
        f["q0"], f["k0"], f["v0"] = self.split(f["y0"], self.w1, H, H, H)
        o, _ = self.lin.step(f["q0"][:, 0], f["k0"][:, 0], f["v0"][:, 0], self.ld, state)
        f["o0"] = o[:, None]
        f["x1"] = f["x0"] + f["o0"].flatten(2)
        f["y1"], *_ = self.norm.forward(f["x1"], self.nw[1], self.nb[1])
        f["q1"], f["k1"], f["v1"] = self.split(f["y1"], self.w2, H, HKV, HKV)
        f["o1"] = self.win.step(f["q1"][:, 0], f["k1"][:, 0], f["v1"][:, 0], k, v, pos)[:, None]
        f["x2"] = f["x1"] + f["o1"].flatten(2)
        return f


def _x(L, dtype, seed=0):
    return torch.randn((B, L, WIDTH), generator=torch.Generator().manual_seed(seed)).to(TYPE[dtype]).cuda()


def _live(t, lens):
    return torch.arange(t.shape[1])[None] < torch.tensor(lens)[:, None]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_and_tokens(dtype):
    s, L, lens, S, n = Stack(dtype), 150, [150, 97, 1], 60, 40
    say(f"stack {dtype}: a prompt and {n} tokens")
    f = s.forward(_x(L, dtype), _i32(lens))
    state = f["state"]
    k, v = (torch.full((B, S, HKV, D), float("nan"), dtype=s.T, device="cuda") for _ in range(2))
    s.win.append(f["k1"], f["v1"], k, v, lens=_i32(lens))
    pos, tokens, steps = _i32(lens), _x(n, dtype, 1), []
    for t in range(n):
        steps.append(s.step(tokens[:, t], state, k, v, pos))
        pos += 1
    # every call against the reference of what the calls were given so far
    for b, m in enumerate(lens):
        whole = {x: torch.cat([f[x][b:b + 1, :m], *(t[x][b:b + 1] for t in steps)], 1) for x in steps[0]}
        d = {x: _f64(t) for x, t in whole.items()}
        for i in "01":
            want, bound = layer_norm_ref.forward(d["x" + i], _f64(s.nw[int(i)]), _f64(s.nb[int(i)]), EPS, dtype)
            check("norm " + i, whole["y" + i], want["y"], bound["y"])
        (want, last), (bound, el) = linear_ref.walk(d["q0"], d["k0"], d["v0"], _f64(s.ld), [m + n], None, D ** -0.5, dtype)
        check("linear", whole["o0"], want, bound)
        check("state", state[b:b + 1], last, el)
        want, bound, _ = window_ref.forward(d["q1"], d["k1"], d["v1"], s.win.cfg)
        check_window("window", whole["o1"].cpu(), want["out"], bound["out"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient(dtype):
    s, L, lens = Stack(dtype), 150, [150, 97, 1]
    say(f"stack {dtype}: the gradient")
    f, dx2 = s.forward(_x(L, dtype), _i32(lens)), _x(L, dtype, 2)
    b = s.backward(f, dx2, _i32(lens))
    df, db = ({n: _f64(t) for n, t in m.items()} for m in (f, b))
    want, bound = window_ref.backward(df["q1"], df["k1"], df["v1"], db["do1"], s.win.cfg, None, lens)
    for n in ("dq", "dk", "dv"):
        check_window("window " + n, b[n + "1"].cpu(), want[n], bound[n])
    want, bound = linear_ref.backward(df["q0"], df["k0"], df["v0"], _f64(s.ld), lens, None, db["do0"], None, D ** -0.5, dtype)
    for n in ("dq", "dk", "dv"):
        check("linear " + n, b[n + "0"], want[n], bound[n])
    for i in "01":
        want, bound = layer_norm_ref.backward(df["x" + i], db["dy" + i], df["mean" + i], df["rstd" + i], _f64(s.nw[int(i)]), dtype)
        for n, t in (("dx", "dn"), ("dweight", "dw"), ("dbias", "db")):
            check(f"norm {i} {n}", b[t + i], want[n], bound[n])
    # padding has a gradient of its own residual alone
    dead = ~_live(dx2, lens).cuda()
    assert torch.equal(b["dx0"][dead], dx2[dead]) and not f["o0"][dead].any() and not f["o1"][dead].any()


def _equal(got, want):
    return all(torch.equal(got[n], want[n]) for n in want)


def test_two_streams():
    """Two stacks' passes on two streams at once are those of one stream, bit for bit."""
    s, x = Stack("bf16"), [_x(700, "bf16", i) for i in range(2)]
    say("stack: two streams")
    want = [(lambda f: {**f, **s.backward(f, t)})(s.forward(t)) for t in x]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in x], []
    for _ in range(3):
        got = []
        for t, st in zip(x, streams):
            with torch.cuda.stream(st):
                f = s.forward(t)
                got.append({**f, **s.backward(f, t)})
        torch.cuda.synchronize()
        assert all(_equal(a, b) for a, b in zip(got, want))


def test_captured():
    """Forward and gradient in one graph, and tokens in another, captured while eager results of the same tensors
    live; replays with other inputs, interleaved, are the eager calls' bits."""
    s, lens = Stack("bf16"), _i32([150, 97, 1])
    say("stack: captured")
    x, tok = _x(150, "bf16"), _x(1, "bf16", 1)[:, 0].contiguous()
    run = lambda: (lambda f: {**f, **s.backward(f, x, lens)})(s.forward(x, lens))  # noqa: E731
    eager = run()
    state, pos = eager["state"].clone(), lens.clone()
    k, v = (torch.zeros((B, 60, HKV, D), dtype=s.T, device="cuda") for _ in range(2))
    s.win.append(eager["k1"], eager["v1"], k, v, lens=lens)
    s.step(tok, state.clone(), k.clone(), v.clone(), pos)
    state2, k2, v2, pos2 = (t.clone() for t in (state, k, v, pos))
    whole, token = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(whole):
        got = run()
    with torch.cuda.graph(token):
        one = s.step(tok, state2, k2, v2, pos2)
        pos2.add_(1)
    for i in range(4):
        x.mul_(1.5 if i % 2 else 0.75)
        tok.copy_(x[:, i])
        whole.replay()
        token.replay()
        want = s.step(tok, state, k, v, pos)
        pos += 1
        torch.cuda.synchronize()
        assert _equal(got, run()) and _equal(one, want), i
        assert all(torch.equal(a, b) for a, b in ((state, state2), (k, k2), (v, v2), (pos, pos2))), i
