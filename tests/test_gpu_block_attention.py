"""GPU: block selection and the attention over selected blocks against the
64-bit reference, within bounds derived there."""
import numpy as np
import pytest

from scale_gla_layer_amd.config import BlockAttentionConfig, RecurrenceConfig
from tests import block_ref as ref
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _type(dtype):
    return _torch().bfloat16 if dtype == "bf16" else _torch().float32


def _op(cfg):
    from scale_gla_layer_amd.runner import DeviceBlockAttention
    return DeviceBlockAttention(cfg)


def _host(t):
    return t.double().cpu().numpy()


def _i32(a):
    return None if a is None else _torch().tensor(np.asarray(a), dtype=_torch().int32, device="cuda")


def _inputs(cfg, B, L, S, seed):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(n, generator=g).to(_type(cfg.dtype)).cuda()  # noqa: E731
    return {"q": r(B, L, cfg.heads_q, cfg.d_k), "k": r(B, S, cfg.heads_kv, cfg.d_k), "v": r(B, S, cfg.heads_kv, cfg.d_v),
            "dout": r(B, L, cfg.heads_q, cfg.d_v)}


def _check(name, got, want, bound):
    g = _host(got)
    fine = np.isfinite(want)
    assert np.array_equal(g[~fine], want[~fine]), f"{name}: infinities"
    assert np.all(np.isfinite(g[fine])), f"{name}: not finite"
    off = np.abs(g[fine] - want[fine])
    b = bound[fine] if bound.shape == want.shape else bound
    worst = float(np.max(off / np.maximum(b, 1e-300) * (off > 0), initial=0))
    assert worst <= 1, f"{name}: {worst:.2f} of its bound"
    say(f"{name}: {worst:.2f} of its bound")


def _case(cfg, B, L, S=None, start=None, lens=None, sel=None, seed=0, grad=True):
    S = L if S is None else S
    say(f"{cfg} B={B} L={L} S={S} start={start} lens={lens}")
    op, t = _op(cfg), _inputs(cfg, B, L, S, seed)
    h = {n: _host(x) for n, x in t.items()}
    ds, dl = _i32(start), _i32(lens)
    means = op.means(t["k"], dl)
    want = ref.means(h["k"], cfg.block, lens)
    # 64 terms in 64 bits, one rounding to 32
    _check("means", means, want, 1.01 * ref.U * np.abs(want) + 1e-16)
    mine = op.select(t["q"], means, ds, dl)
    chosen = ref.select(h["q"], _host(means), cfg, means.shape[2] * cfg.block, start, lens)
    assert np.array_equal(mine.cpu().numpy(), chosen)
    if sel is not None:
        chosen = sel
        mine = _i32(sel)
    out, lse = op.forward(t["q"], t["k"], t["v"], mine, ds, dl)
    want, bound, _ = ref.forward(h["q"], h["k"], h["v"], chosen, cfg, start, lens)
    _check("out", out, want["out"], bound["out"])
    _check("lse", lse, want["lse"], bound["lse"])
    if not grad:
        return
    torch = _torch()
    out = torch.from_numpy(want["out"]).to(_type(cfg.dtype)).cuda().contiguous()
    lse = torch.from_numpy(want["lse"]).float().cuda().contiguous()
    got = op.backward(t["q"], t["k"], t["v"], mine, out, lse, t["dout"], ds, dl)
    want, bound = ref.backward(h["q"], h["k"], h["v"], chosen, h["dout"], cfg, start, lens)
    for name, x in zip(("dq", "dk", "dv"), got):
        _check(name, x, want[name], bound[name])


def _cfg(hq, hkv, dk, dv, block=64, n=6, first=1, recent=2, dtype="bf16", scale=None):
    return BlockAttentionConfig(hq, hkv, dk, dv, block, n, first, recent, scale, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,dk,dv,block,n,L", [
    (4, 1, 64, 64, 64, 4, 1), (4, 2, 64, 64, 32, 4, 2), (2, 2, 128, 128, 64, 5, 333), (6, 2, 80, 96, 32, 6, 401),
    (16, 1, 128, 256, 64, 4, 290), (24, 1, 32, 256, 128, 3, 530), (5, 1, 8, 8, 32, 3, 200), (12, 4, 128, 64, 128, 4, 700),
    (40, 2, 64, 128, 64, 3, 260)])
def test_training(hq, hkv, dk, dv, block, n, L, dtype):
    _case(_cfg(hq, hkv, dk, dv, block, n, dtype=dtype), 2, L, seed=L)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,dk,dv,block,n,B,L,lens", [
    (8, 8, 64, 64, 32, 4, 26, 330, True), (16, 4, 128, 128, 64, 4, 16, 270, False), (24, 8, 80, 96, 32, 6, 16, 171, True),
    (64, 4, 128, 256, 64, 4, 7, 150, False), (40, 2, 64, 128, 128, 3, 4, 277, True), (32, 8, 128, 64, 128, 2, 10, 210, True),
    (16, 1, 32, 256, 64, 20, 3, 1400, False)])
def test_enough_queries_to_share_keys(hq, hkv, dk, dv, block, n, B, L, lens, dtype):
    """At least 4096 tiles: workgroups of 15 tiles (of 3 for wide fp32 heads) share keys and values."""
    cfg = _cfg(hq, hkv, dk, dv, block, n, min(1, n - 2), 2, dtype)
    rng = np.random.default_rng(L)
    if lens:
        start = rng.integers(0, 60, B)
        _case(cfg, B, L, S=L + 77, start=start, lens=np.minimum(start + rng.integers(0, 2 * L, B), L + 60), seed=L)
    else:
        _case(cfg, B, L, seed=L)


def test_enough_queries_with_any_selection():
    cfg = _cfg(16, 16, 64, 64, 32, 8)
    rng = np.random.default_rng(14)
    B, L = 16, 260
    sel = rng.integers(-2, 10, (B, 16, L, 8))
    sel[rng.random(sel.shape) < 0.1] = 2 ** 31 - 1
    sel[rng.random(sel.shape) < 0.1] = -2 ** 31
    sel[0, 0, :100] = -1
    sel[0, 1, :100] = sel[0, 1, :100, :1]
    _case(cfg, B, L, sel=sel.astype(np.int32), seed=9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_any_selection_of_single_queries(dtype):
    cfg = _cfg(12, 3, 64, 80, 32, 8, dtype=dtype)
    rng = np.random.default_rng(15)
    B, S = 5, 300
    sel = rng.integers(-2, 12, (B, 3, 1, 8))
    sel[0, 0], sel[1, 1, 0, 3:] = -1, sel[1, 1, 0, 2]
    sel[2, 2, 0, 1], sel[3, 0, 0, 0] = 2 ** 31 - 1, -2 ** 31
    _case(cfg, B, 1, S=S, start=[299, 150, 64, 0, -1], lens=[300, 151, 300, 1, 300], sel=sel.astype(np.int32), seed=16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,dk,dv,block,n,B,L", [
    (4, 4, 64, 64, 32, 4, 8, 520), (8, 4, 128, 128, 64, 4, 8, 300), (12, 4, 80, 96, 32, 6, 8, 171),
    (64, 4, 128, 256, 64, 4, 2, 150), (40, 2, 64, 128, 128, 3, 1, 277), (16, 4, 128, 64, 128, 2, 4, 290),
    (8, 2, 32, 256, 64, 20, 1, 2100)])
def test_many_queries(hq, hkv, dk, dv, block, n, B, L, dtype):
    """Some thousand tiles, three a workgroup; padding and chunks among them."""
    cfg = _cfg(hq, hkv, dk, dv, block, n, min(1, n - 2), 2, dtype)
    _case(cfg, B, L, seed=L)
    rng = np.random.default_rng(L)
    lens = rng.integers(0, L + 1, B)
    _case(cfg, B, L, lens=lens, seed=L + 1)
    start = rng.integers(0, 100, B)
    _case(cfg, B, L, S=L + 77, start=start, lens=np.minimum(start + L, L + 60), seed=L + 2)


def test_many_queries_with_any_selection():
    cfg = _cfg(8, 4, 64, 64, 32, 8)
    rng = np.random.default_rng(13)
    B, L = 8, 260
    sel = rng.integers(-2, 10, (B, 4, L, 8))
    sel[rng.random(sel.shape) < 0.1] = 2 ** 31 - 1
    sel[rng.random(sel.shape) < 0.1] = -2 ** 31
    sel[0, 0, :100] = -1
    sel[0, 1, :100] = sel[0, 1, :100, :1]
    _case(cfg, B, L, sel=sel.astype(np.int32), seed=9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[300, 129, 64, 1], [0, 300, 7, 250]])
def test_padded_batches(lens, dtype):
    _case(_cfg(6, 2, 64, 96, 32, 5, dtype=dtype), 4, 300, lens=lens, seed=5)


@pytest.mark.parametrize("n,first,recent", [(1, 0, 1), (2, 1, 1), (3, 0, 3), (64, 1, 2), (8, 8 - 1, 1)])
def test_kinds_of_selection(n, first, recent):
    _case(_cfg(4, 2, 64, 64, 32, n, first, recent), 2, 500, seed=n)


@pytest.mark.parametrize("start,lens,L", [([100, 0, 699], [400, 37, 700], 40), ([-5, 690, 3], None, 20),
                                          ([2 ** 31 - 1, -2 ** 31, 0], [700, 700, -3], 9), ([650, 10, 0], [651, 11, 1], 1)])
def test_chunks_of_a_cache(start, lens, L):
    _case(_cfg(8, 2, 64, 64, 64, 4), 3, L, S=700, start=start, lens=lens, seed=7)


def test_any_contents_of_the_selection_are_safe():
    cfg = _cfg(4, 2, 64, 64, 32, 8)
    rng = np.random.default_rng(3)
    B, L = 2, 260
    sel = rng.integers(-2, 10, (B, 2, L, 8))
    sel[rng.random(sel.shape) < 0.1] = 2 ** 31 - 1
    sel[rng.random(sel.shape) < 0.1] = -2 ** 31
    sel[0, 0, :100] = -1  # rows without a block
    sel[0, 1, :100] = sel[0, 1, :100, :1]  # the same index again and again
    _case(cfg, B, L, sel=sel.astype(np.int32), seed=9)


def test_selection_over_many_blocks_and_among_equals():
    """More blocks than are scored at once, and blocks whose scores are equal."""
    torch = _torch()
    cfg = _cfg(4, 2, 64, 64, 32, 7, 2, 2)
    S, B, L = 32 * 1301, 2, 21
    g = torch.Generator().manual_seed(4)
    q = torch.randn((B, L, 4, 64), generator=g).to(torch.bfloat16).cuda()
    means = torch.randn((B, 2, 1301, 64), generator=g).cuda()
    start = np.array([S - 21, 32 * 700 + 3])
    got = _op(cfg).select(q, means, _i32(start))
    assert np.array_equal(got.cpu().numpy(), ref.select(_host(q), _host(means), cfg, S, start))
    few = torch.randn((B, 2, 3, 64), generator=g).cuda()
    means = few[:, :, torch.randint(0, 3, (1301,), generator=g).cuda()].contiguous()
    got = _op(cfg).select(q, means, _i32(start))
    assert np.array_equal(got.cpu().numpy(), ref.select(_host(q), _host(means), cfg, S, start))
    same = means[:, :, :1].expand_as(means).contiguous()
    got = _op(cfg).select(q, same, _i32(start)).cpu().numpy()
    assert np.array_equal(got, ref.select(_host(q), _host(same), cfg, S, start))


def test_special_scores():
    """A NaN ranks as minus infinity; infinities rank at the ends."""
    torch = _torch()
    cfg = _cfg(1, 1, 64, 64, 32, 4, 1, 1)
    means = torch.zeros(1, 1, 9, 64, device="cuda")
    means[0, 0, :, 0] = torch.tensor([0.0, 5.0, float("nan"), -1.0, float("inf"), -2.0, -float("inf"), 4.0, 0.0])
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    got = _op(cfg).select(q, means, _i32([8 * 32]))
    assert got.flatten().tolist() == [0, 1, 4, 8]
    means[0, 0, 1:8, 0] = float("nan")
    assert _op(cfg).select(q, means, _i32([8 * 32])).flatten().tolist() == [0, 1, 2, 8]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_and_what_lies_around_them(dtype):
    """Tensors in one wide projection and head-major layouts; elements outside an output's view stay."""
    torch = _torch()
    cfg = _cfg(4, 2, 64, 96, 32, 4, dtype=dtype)
    B, L = 2, 150
    op, t = _op(cfg), _inputs(cfg, B, L, L, 6)
    means = op.means(t["k"])
    sel = op.select(t["q"], means)
    out, lse = op.forward(t["q"], t["k"], t["v"], sel)
    grads = op.backward(t["q"], t["k"], t["v"], sel, out, lse, t["dout"])
    wide = lambda x: torch.full((B, L + 2, x.shape[2] + 1, x.shape[3] + 16), float("nan"), dtype=x.dtype,  # noqa: E731
                                device="cuda")[:, 1:L + 1, :-1, 8:-8]
    major = lambda x: torch.empty((x.shape[2], B, L, x.shape[3]), dtype=x.dtype, device="cuda").permute(1, 2, 0, 3)  # noqa: E731
    for make in (wide, major):
        u = {n: make(x).copy_(x) for n, x in t.items()}
        assert torch.equal(op.means(u["k"]), means) and torch.equal(op.select(u["q"], means), sel)
        o = make(out)
        o2, lse2 = op.forward(u["q"], u["k"], u["v"], sel, out=o)
        assert o2 is o and torch.equal(o, out) and torch.equal(lse2, lse)
        d = [make(x) for x in grads]
        op.backward(u["q"], u["k"], u["v"], sel, o, lse, u["dout"], dq=d[0], dk=d[1], dv=d[2])
        for a, b in zip(d, grads):
            assert torch.equal(a, b)
        for x in (o, *d):
            if make is wide:
                x.fill_(float("nan"))
                assert bool(x._base.isnan().all())


def test_what_lies_behind_the_sequences_has_no_influence():
    torch = _torch()
    cfg = _cfg(8, 2, 64, 64, 64, 4)
    B, L, lens = 3, 300, [300, 70, 1]
    op, t = _op(cfg), _inputs(cfg, B, L, L, 8)
    dl = _i32(lens)

    def run():
        means = op.means(t["k"], dl)
        sel = op.select(t["q"], means, lens=dl)
        out, lse = op.forward(t["q"], t["k"], t["v"], sel, lens=dl)
        return [means, sel, out, lse, *op.backward(t["q"], t["k"], t["v"], sel, out, lse, t["dout"], lens=dl)]

    want = run()
    behind = torch.arange(L, device="cuda")[None] >= dl[:, None]
    for value in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        for n in t:
            t[n][behind] = value
        for a, b in zip(run(), want):
            assert torch.equal(a, b)
    for x in want[2], want[4], want[5], want[6]:
        assert bool((x[behind] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,dk,dv,block", [(8, 2, 64, 64, 64), (3, 1, 128, 256, 32), (20, 1, 80, 128, 128)])
def test_steps(hq, hkv, dk, dv, block, dtype):
    """Steps over caches that hold anything behind their tokens, past the end of blocks, against the reference."""
    torch = _torch()
    cfg = _cfg(hq, hkv, dk, dv, block, 4, dtype=dtype)
    B, S, n = 3, 5 * block + 7, 6
    op, t = _op(cfg), _inputs(cfg, B, S, S, 10)
    pos = np.array([block - 3, 4 * block - 1, 5 * block - 2])
    behind = torch.arange(S, device="cuda")[None] >= _i32(pos)[:, None]
    k, v = t["k"].clone(), t["v"].clone()
    k[behind], v[behind] = float("nan"), float("nan")
    means = op.means(k, _i32(pos))
    kr, vr, mr = _host(t["k"]), _host(t["v"]), None
    for s in range(n):
        row, at = torch.arange(B, device="cuda"), _i32(pos).long()
        q, kt, vt = t["q"][:, s].contiguous(), t["k"][row, at], t["v"][row, at]
        out = op.step(q, kt, vt, k, v, means, _i32(pos))
        mr = ref.means(kr, block, pos + 1)
        whole = np.arange(1, means.shape[2] + 1) * block <= pos[:, None] + 1
        sel = ref.select(_host(q)[:, None], mr.astype(np.float32).astype(np.float64), cfg, S, pos)
        want, bound, _ = ref.forward(_host(q)[:, None], kr, vr, sel, cfg, pos)
        _check("out", out, want["out"][:, 0], bound["out"][:, 0])
        got = _host(means).transpose(0, 2, 1, 3)[whole]
        assert np.all(np.abs(got - mr.transpose(0, 2, 1, 3)[whole]) <= 1.01 * ref.U * np.abs(got) + 1e-16)
        pos = pos + 1
    filled = torch.arange(S, device="cuda")[None] < _i32(pos)[:, None]
    assert torch.equal(k[filled], t["k"][filled]) and torch.equal(v[filled], t["v"][filled])
    assert bool(k[~filled].isnan().all()) and bool(v[~filled].isnan().all())
    # positions outside the caches: nothing is written, the output row is zero
    before = k.nan_to_num().clone()
    out = op.step(q, kt, vt, k, v, means, _i32([-1, S, 2 ** 31 - 1]))
    assert bool((out == 0).all()) and torch.equal(k.nan_to_num(), before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("blocks", [129, 700])
def test_steps_over_long_caches(blocks, dtype):
    """More blocks than one workgroup scores, and than one piece of the choice holds; equal blocks, which go to the
    lower index, and positions outside."""
    torch = _torch()
    cfg = _cfg(6, 2, 64, 64, 32, 9, dtype=dtype)
    B, S = 6, 32 * blocks - 3
    op, t = _op(cfg), _inputs(cfg, B, 1, S, 22)
    k, v = t["k"], t["v"]
    k[2, :] = k[2, :32].repeat(blocks, 1, 1)[:S]  # the same mean in every block
    k[3, 32 * 64:] = k[3, 32 * 64:32 * 65].repeat(blocks, 1, 1)[:S - 32 * 64]
    pos = np.array([S - 1, 32 * 128 - 1, S - 2, S - 40, -1, 31])
    row, at = torch.arange(B, device="cuda"), _i32(np.maximum(pos, 0)).long()
    q, kt, vt = t["q"][:, 0].contiguous(), k[row, at], v[row, at]
    means = op.means(k, _i32(np.maximum(pos, 0)))
    want_means = op.means(k, _i32(pos + 1))
    sel = ref.select(_host(q)[:, None], _host(want_means), cfg, S, pos)
    want, bound, _ = ref.forward(_host(q)[:, None], _host(k), _host(v), sel, cfg, pos)
    k0, v0 = k.clone(), v.clone()
    out = op.step(q, kt, vt, k, v, means, _i32(pos))
    _check("out", out, want["out"][:, 0], bound["out"][:, 0])
    assert bool((out[4] == 0).all()) and torch.equal(k, k0) and torch.equal(v, v0)
    assert torch.equal(means, want_means)


def test_more_blocks_than_shared_tiles_hold():
    """A cache of so many blocks that tiles do not share them, against its part that the selection names."""
    torch = _torch()
    cfg = _cfg(16, 1, 64, 64, 32, 6)
    B, L, S = 1, 131, 32 * 16385
    op, t = _op(cfg), _inputs(cfg, B, L, S, 23)
    rng = np.random.default_rng(24)
    sel = np.sort(np.stack([rng.permutation(8)[:6] for _ in range(L)]))[None, None]
    start = _i32([S - L])
    out, lse = op.forward(t["q"], t["k"], t["v"], _i32(sel), start)
    grads = op.backward(t["q"], t["k"], t["v"], _i32(sel), out, lse, t["dout"], start)
    # every query by itself, at the last position of the eight blocks
    q, do = (_host(t[n])[0][:, None] for n in ("q", "dout"))
    k, v = (np.repeat(_host(t[n][:, :256]), L, axis=0) for n in "kv")
    last, rows = np.full(L, 255), np.moveaxis(sel[0], 1, 0)[:, :, None]
    want, bound, _ = ref.forward(q, k, v, rows, cfg, last)
    _check("out", out[0][:, None], want["out"], bound["out"])
    _check("lse", lse[0].t()[:, :, None], want["lse"], bound["lse"])
    want, bound = ref.backward(q, k, v, rows, do, cfg, last)
    _check("dq", grads[0][0][:, None], want["dq"], bound["dq"])
    for name, g in zip(("dk", "dv"), grads[1:]):
        _check(name, g[0, :256], want[name].sum(0), bound[name].sum(0))
        assert bool((g[0, 256:] == 0).all())


def test_means_of_a_growing_cache():
    torch = _torch()
    cfg = _cfg(4, 2, 64, 64, 32, 4)
    op, t = _op(cfg), _inputs(cfg, 2, 200, 200, 11)
    done, now = [70, 0], [199, 32]
    means = op.means(t["k"], _i32(done))
    means[0, :, 0] = 7.0  # a block that ended before: kept
    op.means(t["k"], _i32(now), start_from=_i32(done), means=means)
    want = op.means(t["k"], _i32(now))
    assert bool((means[0, :, 0] == 7.0).all())
    want[0, :, 0] = 7.0
    assert torch.equal(means, want)


@pytest.mark.parametrize("L,dv", [(3, 64), (300, 64), (2100, 256)])
def test_captured_calls_share_nothing(L, dv):
    torch = _torch()
    cfg = _cfg(8, 2, 64, dv, 64, 4) if L < 2000 else _cfg(64, 2, 128, dv, 64, 4)
    op = _op(cfg)
    sets = []
    for seed in (20, 21):
        t = _inputs(cfg, 2, L, L, seed)
        pos, kt = _i32([1, 2]), t["k"][:, :1].squeeze(1).clone()
        vt, qt = t["v"][:, 0].clone(), t["q"][:, 0].clone()

        def call(t=t, pos=pos, kt=kt, vt=vt, qt=qt):
            means = op.means(t["k"])
            sel = op.select(t["q"], means)
            out, lse = op.forward(t["q"], t["k"], t["v"], sel)
            grads = op.backward(t["q"], t["k"], t["v"], sel, out, lse, t["dout"])
            return [means, sel, out, lse, *grads, op.step(qt, kt, vt, t["k"].clone(), t["v"].clone(), means, pos)]

        eager = call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        sets.append((graph, got, eager, call))
    for _ in range(3):
        for graph, got, eager, call in sets:
            for x in got:
                x.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(call(), eager))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, eager))


def test_another_stream():
    torch = _torch()
    cfg = _cfg(8, 2, 64, 64, 32, 4)
    op, t = _op(cfg), _inputs(cfg, 2, 500, 500, 12)

    def call():
        sel = op.select(t["q"], op.means(t["k"]))
        out, lse = op.forward(t["q"], t["k"], t["v"], sel)
        return [out, lse, *op.backward(t["q"], t["k"], t["v"], sel, out, lse, t["dout"])]

    want = call()
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    for _ in range(3):
        with torch.cuda.stream(side):
            got.append(call())
        got.append(call())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_refusals():
    torch = _torch()
    cfg = _cfg(4, 2, 64, 64, 32, 4)
    op, t = _op(cfg), _inputs(cfg, 2, 40, 40, 13)
    means = op.means(t["k"])
    sel = op.select(t["q"], means)
    for kw in (dict(q=t["q"].float()), dict(k=t["k"][:, :, :1]), dict(v=t["v"].cpu()), dict(sel=sel.long()),
               dict(sel=sel[:, :, :-1]), dict(start=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(lens=torch.zeros(2, device="cuda")), dict(q=t["q"].transpose(2, 3).contiguous().transpose(2, 3)),
               dict(out=t["q"][:, :1].expand(2, 40, 4, 64)), dict(lse=torch.zeros(2, 40, 4, device="cuda"))):
        with pytest.raises(ValueError):
            op.forward(**{**{n: t[n] for n in "qkv"}, "sel": sel, **kw})
    odd = torch.zeros(2 * 40 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(2, 40, 2, 64)
    with pytest.raises(ValueError, match="multiples of 16 bytes"):
        op.means(odd)
    with pytest.raises(ValueError):
        op.select(t["q"], means[:, :1])
    with pytest.raises(ValueError):
        op.step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["k"], t["v"], means, torch.zeros(2, device="cuda"))


def test_a_stack_of_both_operators():
    """A recurrence feeding an attention, as a hybrid model's two mixers: a prefill of a prompt, then steps with
    both states, against one pass over the whole sequence; and the training pass's gradients against the
    64-bit reference through the projections between."""
    torch = _torch()
    from scale_gla_layer_amd.runner import DeviceRecurrence
    from tests import recurrence_ref
    B, L, D, cut = 2, 200, 128, 150
    acfg, rcfg = _cfg(4, 2, 32, 32, 32, 4, dtype="f32"), RecurrenceConfig(D, "norm", 8.0, "f32")
    att, rec = _op(acfg), DeviceRecurrence(rcfg)
    g = torch.Generator().manual_seed(30)
    x, z = (torch.randn((B, L, D), generator=g).cuda() for _ in range(2))
    W = (torch.randn((D, 4 * 32 + 2 * 32 + 2 * 32), generator=g) * D ** -0.5).cuda()

    def qkv(y):
        p = y @ W
        return (p[..., :128].unflatten(-1, (4, 32)), p[..., 128:192].unflatten(-1, (2, 32)),
                p[..., 192:].unflatten(-1, (2, 32)))

    y, _ = rec.forward(x, z)
    q, k, v = qkv(y)
    sel = att.select(q, att.means(k))
    out, lse = att.forward(q, k, v, sel)
    # streaming
    yp, h = rec.forward(x[:, :cut], z[:, :cut])
    qp, kp, vp = qkv(yp)
    ck, cv = torch.zeros((B, L, 2, 32), device="cuda"), torch.zeros((B, L, 2, 32), device="cuda")
    ck[:, :cut], cv[:, :cut] = kp, vp
    lens = _i32([cut, cut])
    means = att.means(ck, lens)
    s = att.select(qp, means, lens=lens)
    op, _ = att.forward(qp, ck, cv, s, lens=lens)
    parts, pos = [op], _i32([cut, cut])
    for t in range(cut, L):
        yt, h = rec.step(x[:, t], z[:, t], h)
        qt, kt, vt = qkv(yt)
        parts.append(att.step(qt, kt, vt, ck, cv, means, pos)[:, None])
        pos += 1
    # two orders of the same 32-bit sums; a selection that hangs on their difference would show as a whole block
    assert torch.allclose(torch.cat(parts, 1), out, rtol=0, atol=1e-4 * float(out.abs().max()))
    # training
    dout = torch.randn(out.shape, generator=g).cuda()
    dq, dk, dv = att.backward(q, k, v, sel, out, lse, dout)
    dp = torch.cat((dq.flatten(2), dk.flatten(2), dv.flatten(2)), -1)
    dx, dz, _, _ = rec.backward(x, z, dp @ W.T)
    hx, hz, hW = _host(x), _host(z), _host(W)
    hy = recurrence_ref.forward(hx, hz, np.zeros(D), 8.0, "norm")[0]["y"]
    hp = hy @ hW
    hq, hk, hv = hp[..., :128].reshape(B, L, 4, 32), hp[..., 128:192].reshape(B, L, 2, 32), hp[..., 192:].reshape(B, L, 2, 32)
    hs = ref.select(hq, ref.means(hk, 32), acfg, L)
    assert np.array_equal(hs, sel.cpu().numpy())
    gq = ref.backward(hq, hk, hv, hs, _host(dout), acfg)[0]
    hd = np.concatenate([gq[n].reshape(B, L, -1) for n in ("dq", "dk", "dv")], -1) @ hW.T
    want = recurrence_ref.backward(hx, hz, hd, np.zeros(D), 8.0, "norm")[0]
    for name, got in (("dx", dx), ("dz", dz)):
        # errors of 32-bit sums of a few hundred terms, three products deep: 2^-24 * 1000
        off = np.linalg.norm(_host(got) - want[name]) / np.linalg.norm(want[name])
        say(f"{name} relative error {off:.1e}")
        assert off < 1000 * ref.U
