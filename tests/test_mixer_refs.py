"""CPU: the 64-bit references of layer norm, linear attention and window attention against formulas of their own and
differences."""
import pytest
import torch

from scale_gla_layer_amd.config import WindowAttentionConfig
from tests import layer_norm_ref, linear_ref, window_ref


def _g(seed):
    return torch.Generator().manual_seed(seed)


def _differences(f, x, n, seed, h=1e-5):
    """[(index, central difference of f at it)] for n elements of x."""
    at = torch.randperm(x.numel(), generator=_g(seed))[:n].tolist()
    out = []
    for i in at:
        y = x.flatten().clone()
        y[i] += h
        up = f(y.view_as(x))
        y[i] -= 2 * h
        out.append((i, (up - f(y.view_as(x))) / (2 * h)))
    return out


def _agree(grad, diffs, tol=1e-6):
    flat = grad.flatten()
    size = max(1.0, float(flat.abs().max()))
    for i, d in diffs:
        assert abs(float(flat[i] - d)) <= tol * size, (i, float(flat[i]), float(d))


def test_layer_norm():
    g = _g(1)
    x, dy = torch.randn((2, 3, 7), generator=g, dtype=torch.float64), torch.randn((2, 3, 7), generator=g, dtype=torch.float64)
    w, b = torch.randn(7, generator=g, dtype=torch.float64), torch.randn(7, generator=g, dtype=torch.float64)
    got, _ = layer_norm_ref.forward(x, w, b, 1e-5, "f32")
    assert torch.allclose(got["y"], torch.nn.functional.layer_norm(x, (7,), w, b, 1e-5), rtol=1e-12, atol=1e-12)
    grads, _ = layer_norm_ref.backward(x, dy, got["mean"], got["rstd"], w, "f32")
    loss = lambda x_, w_, b_: float((layer_norm_ref.forward(x_, w_, b_, 1e-5, "f32")[0]["y"] * dy).sum())  # noqa: E731
    _agree(grads["dx"], _differences(lambda t: loss(t, w, b), x, 20, 2))
    _agree(grads["dweight"], _differences(lambda t: loss(x, t, b), w, 7, 3))
    _agree(grads["dbias"], _differences(lambda t: loss(x, w, t), b, 7, 4))


@pytest.mark.parametrize("lens", [[6, 6], [6, 2], [0, 5]])
@pytest.mark.parametrize("with_state", [False, True])
def test_linear(lens, with_state):
    g = _g(5)
    B, L, H, dk, dv, scale = 2, 6, 2, 3, 4, 0.7
    r = lambda *n: torch.randn(n, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = r(B, L, H, dk), r(B, L, H, dk), r(B, L, H, dv), r(B, L, H, dv)
    lg = torch.tensor([-0.1, -0.6], dtype=torch.float64)
    S, dS = (r(B, H, dk, dv), r(B, H, dk, dv)) if with_state else (None, r(B, H, dk, dv))
    run = lambda q_, k_, v_, s_: linear_ref.walk(q_, k_, v_, lg, lens, s_, scale, "f32")[0]  # noqa: E731
    out, last = run(q, k, v, S)
    # the sum itself
    for b, n in enumerate(lens):
        for h in range(H):
            for t in range(L):
                want = torch.zeros(dv, dtype=torch.float64)
                if t < n:
                    for s in range(t + 1):
                        want += scale * torch.exp(lg[h] * (t - s)) * (q[b, t, h] @ k[b, s, h]) * v[b, s, h]
                    if with_state:
                        want += scale * torch.exp(lg[h] * (t + 1)) * (q[b, t, h] @ S[b, h])
                assert torch.allclose(out[b, t, h], want, atol=1e-12)
    loss = lambda *a: float((run(*a)[0] * do).sum() + (run(*a)[1] * dS).sum())  # noqa: E731
    grads, _ = linear_ref.backward(q, k, v, lg, lens, S, do, dS, scale, "f32")
    _agree(grads["dq"], _differences(lambda t: loss(t, k, v, S), q, 20, 6))
    _agree(grads["dk"], _differences(lambda t: loss(q, t, v, S), k, 20, 7))
    _agree(grads["dv"], _differences(lambda t: loss(q, k, t, S), v, 20, 8))
    if with_state:
        _agree(grads["dstate"], _differences(lambda t: loss(q, k, v, t), S, 20, 9))


def test_linear_without_memory():
    """gamma = 0: each token on its own; the state is the last token's."""
    g = _g(11)
    q, k, v = (torch.randn((1, 3, 1, 2), generator=g, dtype=torch.float64) for _ in range(3))
    (out, last), _ = linear_ref.walk(q, k, v, torch.tensor([-float("inf")], dtype=torch.float64), [3], None, 1.0, "f32")
    assert torch.allclose(out, (q * k).sum(3, keepdim=True) * v)
    assert torch.allclose(last[0, 0], torch.outer(k[0, 2, 0], v[0, 2, 0]))


@pytest.mark.parametrize("window,n_sink,start,lens", [(3, 0, None, None), (2, 2, [0, 3], [9, 6]), (20, 0, [1, -2], None),
                                                      (1, 1, None, [0, 5])])
def test_window(window, n_sink, start, lens):
    g = _g(21)
    B, L, S, hq, hkv, dk, dv = 2, 7, 9, 4, 2, 8, 16
    cfg = WindowAttentionConfig(hq, hkv, dk, dv, window, n_sink, dtype="f32")
    r = lambda *n: torch.randn(n, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = r(B, L, hq, dk), r(B, S, hkv, dk), r(B, S, hkv, dv), r(B, L, hq, dv)
    got, _, _ = window_ref.forward(q, k, v, cfg, start, lens)
    for b in range(B):
        for i in range(L):
            p = i + (start[b] if start else 0)
            n = min(lens[b], S) if lens else S
            for h in range(hq):
                keys = [j for j in range(S) if j <= p and (p - j < window or j < n_sink)] if 0 <= p < n else []
                if not keys:
                    assert (got["out"][b, i, h] == 0).all() and got["lse"][b, h, i] == -torch.inf
                    continue
                s = k[b, keys, h // 2] @ q[b, i, h] * cfg.scale
                assert torch.allclose(got["lse"][b, h, i], torch.logsumexp(s, 0))
                assert torch.allclose(got["out"][b, i, h], torch.softmax(s, 0) @ v[b, keys, h // 2])
    loss = lambda *a: float((window_ref.forward(*a, cfg, start, lens)[0]["out"] * do).sum())  # noqa: E731
    grads, _ = window_ref.backward(q, k, v, do, cfg, start, lens)
    _agree(grads["dq"], _differences(lambda t: loss(t, k, v), q, 25, 22))
    _agree(grads["dk"], _differences(lambda t: loss(q, t, v), k, 25, 23))
    _agree(grads["dv"], _differences(lambda t: loss(q, k, t), v, 25, 24))


def test_window_slots():
    """A rolling cache of n_sink + window slots holds exactly what the next query attends."""
    for S, n_sink, window in ((7, 2, 5), (8, 0, 5), (12, 3, 5)):
        held = {}
        for p in range(40):
            held[window_ref.slot(p, S, n_sink)] = p
            want = [j for j in range(p + 1) if j > p - window or j < n_sink]
            assert set(want) <= set(held.values()) and len(held) <= S
