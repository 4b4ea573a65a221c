"""GPU: layer norm against the 64-bit reference, within bounds derived there: widths around every shape of a row, odd
ones, strided views, special values, graph replays and refusals."""
import pytest
import torch

from scale_gla_layer_amd.config import LayerNormConfig
from tests import layer_norm_ref as ref
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _handle(*a, **k):
    from scale_gla_layer_amd.runner import DeviceLayerNorm
    return DeviceLayerNorm(LayerNormConfig(*a, **k))


def _inputs(B, L, D, dtype, seed=0, shift=0.5, affine=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(n, generator=g)  # noqa: E731
    v = {"x": (r(B, L, D) * 2 + shift).to(TYPE[dtype]), "dy": r(B, L, D).to(TYPE[dtype])}
    v.update(weight=1 + 0.5 * r(D) if affine else None, bias=r(D) if affine else None)
    return v


def _dev(t):
    return None if t is None else t.cuda()


def _f64(t):
    return None if t is None else t.detach().double().cpu()


def check(name, got, want, bound):
    g = _f64(got)
    assert g.shape == want.shape, f"{name}: {tuple(g.shape)}"
    assert torch.isfinite(g).all(), f"{name}: not finite"
    off = (g - want).abs()
    worst = float((off / bound.clamp(min=1e-300) * (off > 0)).max())
    assert worst <= 1, f"{name}: {worst:.2f} of its bound"
    say(f"{name}: {worst:.2f} of its bound")


def _case(B, L, D, dtype, eps=1e-5, affine=True, shift=0.5, views=None):
    say(f"layer norm B={B} L={L} D={D} {dtype} affine={affine} shift={shift}")
    v, h = _inputs(B, L, D, dtype, affine=affine, shift=shift), _handle(D, eps, dtype)
    x, dy, w, b = (_dev(v[n]) for n in ("x", "dy", "weight", "bias"))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    if views:
        x, dy, y, dx = (views(t) for t in (x, dy, y, dx))
    got_y, mean, rstd = h.forward(x, w, b, y=y)
    assert got_y.data_ptr() == y.data_ptr()
    want, bound = ref.forward(_f64(v["x"]), _f64(v["weight"]), _f64(v["bias"]), eps, dtype)
    for n, t in (("y", y), ("mean", mean), ("rstd", rstd)):
        check(n, t, want[n], bound[n])
    _, dw, db = h.backward(x, dy, mean, rstd, w, b, dx=dx)
    want, bound = ref.backward(_f64(v["x"]), _f64(v["dy"]), _f64(mean), _f64(rstd), _f64(v["weight"]), dtype)
    check("dx", dx, want["dx"], bound["dx"])
    assert (dw is None) == (w is None) and (db is None) == (b is None)
    if affine:
        check("dweight", dw, want["dweight"], bound["dweight"])
        check("dbias", db, want["dbias"], bound["dbias"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 3, 7, 8, 64, 65, 127, 128, 129, 256, 257, 511, 512, 513, 1000, 1001, 1024, 1025, 2047,
                               2048, 2049, 4096, 4097, 8191, 8192, 8193, 16383, 16384])
def test_widths(D, dtype):
    _case(2, 5, D, dtype)


@pytest.mark.parametrize("B,L,D,dtype", [(1, 1, 1024, "bf16"), (16, 1, 1024, "bf16"), (1, 4500, 96, "bf16"),
                                         (3, 1500, 1024, "bf16"), (3, 1367, 1001, "f32"), (1, 9001, 8, "f32"),
                                         (2, 1100, 2056, "bf16"), (1, 2100, 4100, "f32"), (5, 7, 9000, "bf16")])
def test_rows(B, L, D, dtype):
    _case(B, L, D, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [40, 1024, 9000])
def test_without_parameters_and_shifted(D, dtype):
    _case(2, 9, D, dtype, affine=False)
    _case(2, 9, D, dtype, shift=1000.0)


def test_one_parameter_alone():
    v, h = _inputs(2, 6, 77, "f32"), _handle(77, dtype="f32")
    x, dy, w, b = (_dev(v[n]) for n in ("x", "dy", "weight", "bias"))
    _, mean, rstd = h.forward(x, w)
    dx, dw, db = h.backward(x, dy, mean, rstd, w)
    assert db is None
    _, _, both = h.backward(x, dy, mean, rstd, w, b)
    want, bound = ref.backward(*(_f64(t) for t in (x, dy, mean, rstd, w)), "f32")
    check("dweight", dw, want["dweight"], bound["dweight"])
    check("dbias", both, want["dbias"], bound["dbias"])
    dx0, dw0, db0 = h.backward(x, dy, mean, rstd, None, b)
    want, bound = ref.backward(*(_f64(t) for t in (x, dy, mean, rstd)), None, "f32")
    assert dw0 is None
    check("dx without weight", dx0, want["dx"], bound["dx"])
    check("dbias without weight", db0, want["dbias"], bound["dbias"])


def test_strided_views():
    def wide(t):  # columns of a wider tensor, from an odd element, sequences far apart
        B, L, D = t.shape
        big = torch.full((B, 2 * L, D + 9), float("nan"), dtype=t.dtype, device="cuda")
        view = big[:, 1:2 * L:2, 3:3 + D]
        view.copy_(t)
        return view
    for D, dtype in ((96, "bf16"), (1001, "f32"), (2050, "bf16")):
        _case(3, 17, D, dtype, views=wide)
    _case(3, 17, 64, "f32", views=lambda t: t.transpose(0, 1).contiguous().transpose(0, 1))


def test_in_place():
    for D, dtype in ((96, "bf16"), (4097, "f32"), (9000, "bf16")):
        v, h = _inputs(2, 700, D, dtype), _handle(D, dtype=dtype)
        x, dy, w, b = (_dev(v[n]) for n in ("x", "dy", "weight", "bias"))
        y, mean, rstd = h.forward(x, w, b)
        dx, dw, db = h.backward(x, dy, mean, rstd, w, b)
        x2, dy2 = x.clone(), dy.clone()
        h.forward(x2, w, b, y=x2)
        _, dw2, db2 = h.backward(x, dy2, mean, rstd, w, b, dx=dy2)
        assert torch.equal(x2, y) and torch.equal(dy2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("D,dtype", [(50, "bf16"), (1001, "f32"), (3000, "f32"), (9000, "bf16")])
def test_special_values_stay_in_their_row(D, dtype):
    v, h = _inputs(1, 6, D, dtype), _handle(D, dtype=dtype)
    x, w, b = _dev(v["x"]), _dev(v["weight"]), _dev(v["bias"])
    y, mean, rstd = h.forward(x, w, b)
    x2 = x.clone()
    x2[0, 1, D // 2], x2[0, 3, 0], x2[0, 4] = float("nan"), float("inf"), 3.0
    y2, mean2, rstd2 = h.forward(x2, w, b)
    for r in (0, 2, 5):
        assert torch.equal(y2[0, r], y[0, r]) and mean2[0, r] == mean[0, r] and rstd2[0, r] == rstd[0, r]
    assert y2[0, 1].isnan().all() and not y2[0, 3].isfinite().any()
    # a row of one value: the bias, beside at most 2^-22 of the mean's rounding (3 * 2^-24) times rstd (316)
    assert ((y2[0, 4].float() - b).abs() <= ref.HALF[dtype] * b.abs() + 1e-7).all() and abs(float(mean2[0, 4]) - 3) < 1e-6
    assert abs(float(rstd2[0, 4]) - 1e-5 ** -0.5) < 0.01


def test_bits_repeat_and_graphs():
    v, h = _inputs(3, 1500, 1024, "bf16"), _handle(1024)
    x, dy, w, b = (_dev(v[n]) for n in ("x", "dy", "weight", "bias"))
    want = (*h.forward(x, w, b), *h.backward(x, dy, *h.forward(x, w, b)[1:], w, b))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, mean, rstd = h.forward(x, w, b)
        got = (y, mean, rstd, *h.backward(x, dy, mean, rstd, w, b))
    keep = x.clone()
    for i in range(3):
        x.copy_(keep * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        again = (*h.forward(x, w, b), *h.backward(x, dy, *h.forward(x, w, b)[1:], w, b))
        assert all(torch.equal(p, q) for p, q in zip(got, again)), i
        if i == 0:
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_refusals():
    v, h = _inputs(2, 3, 64, "bf16"), _handle(64)
    x, dy, w, b = (_dev(v[n]) for n in ("x", "dy", "weight", "bias"))
    y, mean, rstd = h.forward(x, w, b)
    for bad in (lambda: h.forward(x[0], w, b), lambda: h.forward(x.float(), w, b), lambda: h.forward(x[..., :63], w, b),
                lambda: h.forward(x, w.bfloat16(), b), lambda: h.forward(x, w, b[:3]), lambda: h.forward(x.cpu(), w, b),
                lambda: h.forward(x, w, b, y=x[:1].expand(2, 3, 64)), lambda: h.forward(x, w, b.cpu()),
                lambda: h.backward(x, dy[:1], mean, rstd, w, b), lambda: h.backward(x, dy, mean[:1], rstd, w, b),
                lambda: h.backward(x, dy, None, rstd, w, b), lambda: h.backward(x[0], dy[0], mean, rstd, w, b),
                lambda: h.forward(x.transpose(1, 2).contiguous().transpose(1, 2), w, b)):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    with pytest.raises((ValueError, RuntimeError)):
        h.forward(x[:0], w, b)
