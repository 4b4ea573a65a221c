"""Sliding-window attention in 64 bits, and bounds on what a computation with 32-bit
sums may be off.

Bounds.  u = 2^-24; h is half a step of the storage type.  A score (a sum of d_k
products, scaled, an exponent after a multiplication and an addition) is off by at
most D = (d_k + 4) u scale sum |q k| + 6 u max |s|, the largest of which in a row,
twice (numerator and normaliser), is the relative error of a softmax weight, with
(n + 32) u for the exponential and the sum over n keys.  For bf16 a weight enters its
product as two bf16 values, which leaves 2^-18 = 64 u of it.  An output is off by that
share of sum p |v| and by half a step of itself.
Gradients: weights come from the stored lse, another 4 u |lse|.  dp (a sum of d_v
products) is off by (d_v + 4) u sum |do v|.  delta: for bf16 it is put right by the
weights' own sum of p dp, so it is off by their share of sum p |dp| + |delta|, and dp's
error; what remains is e = h sum |do o| times the rounding of the weights in
sum p k, 2^-9.  For fp32 it comes from the stored output: (h + (d_v + 4) u) sum |do o|
and the output's error.  The score's gradient p (dp - delta) scale adds the weight's
share and, for bf16, 64 u; the sums over keys or rows add (number of terms) u."""
import torch

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def positions(B, L, S, start=None, lens=None):
    """[B, L], -1 for padding."""
    p = (torch.zeros(B, dtype=torch.int64) if start is None else torch.tensor(start))[:, None] + torch.arange(L)
    n = torch.full((B, 1), S) if lens is None else torch.tensor(lens)[:, None].clamp(max=S)
    return torch.where((p >= 0) & (p < n), p, -1)


def allowed(p, S, window, n_sink):
    """[B, L, S]"""
    j, p = torch.arange(S), p[:, :, None]
    return (j <= p) & ((j > p - window) | (j < n_sink))


def _heads(t):
    return t.transpose(1, 2)


def forward(q, k, v, cfg, start=None, lens=None, p=None):
    """(values, bounds), each {"out", "lse"}, and what the gradients need.  q, k, v in 64 bits, anywhere."""
    B, L, S, G, h = q.shape[0], q.shape[1], k.shape[1], cfg.heads_q // cfg.heads_kv, HALF[cfg.dtype]
    p = positions(B, L, S, start, lens) if p is None else p
    hit = allowed(p, S, cfg.window, cfg.n_sink).to(q.device)[:, None]
    used = hit.any(2)[:, 0, :, None, None]  # what no query attends may be anything
    kk, vv = (_heads(torch.where(used, t, 0.0)).repeat_interleave(G, 1) for t in (k, v))
    qq = torch.where((p >= 0).to(q.device)[:, None, :, None], _heads(q), 0.0)
    s = qq @ kk.transpose(2, 3) * cfg.scale
    size = qq.abs() @ kk.abs().transpose(2, 3) * cfg.scale
    some = hit.any(3, keepdim=True)
    top = torch.where(some, s.masked_fill(~hit, -torch.inf).amax(3, keepdim=True), 0.0)
    e = torch.where(hit, torch.exp(torch.where(hit, s - top, 0.0)), 0.0)
    total = e.sum(3, keepdim=True)
    w = e / torch.where(some, total, 1.0)
    most = torch.where(hit, s.abs(), 0.0).amax(3, keepdim=True)
    off = torch.where(hit, (cfg.d_k + 4) * U * size, 0.0).amax(3, keepdim=True) + 6 * U * most
    share = 2 * off + (hit.sum(3, keepdim=True) + 32) * U
    split = 64 * U if cfg.dtype == "bf16" else 0.0
    out = w @ vv
    eo = (share + split) * (w @ vv.abs())
    lse = torch.where(some, top + torch.log(torch.where(some, total, 1.0)), -torch.inf)[..., 0]
    el = torch.where(some, share + 4 * U * torch.where(some, lse[..., None], 0.0).abs(), 0.0)[..., 0]
    keep = {"w": w, "hit": hit, "share": share, "split": split, "q": qq, "k": kk, "v": vv, "out": out, "eo": eo,
            "lse": torch.where(some[..., 0], lse, 0.0), "live": (p >= 0).to(q.device)}
    return {"out": _heads(out), "lse": lse}, {"out": _heads(eo + h * (out.abs() + eo)), "lse": el}, keep


def backward(q, k, v, dout, cfg, start=None, lens=None):
    _, _, f = forward(q, k, v, cfg, start, lens)
    B, G, h, w = q.shape[0], cfg.heads_q // cfg.heads_kv, HALF[cfg.dtype], f["w"]
    do = torch.where(f["live"][:, None, :, None], _heads(dout), 0.0)
    share = f["share"] + 4 * U * f["lse"][..., None].abs()
    dp = do @ f["v"].transpose(2, 3)
    edp = (cfg.d_v + 4) * U * (do.abs() @ f["v"].abs().transpose(2, 3))
    delta = (do * f["out"]).sum(3, keepdim=True)
    rest = h * (do * f["out"]).abs().sum(3, keepdim=True)
    if cfg.dtype == "bf16":
        edelta = share * ((w * dp.abs()).sum(3, keepdim=True) + delta.abs()) + (w * edp).sum(3, keepdim=True)
    else:
        edelta = rest + (do.abs() * (f["eo"] + (cfg.d_v + 4) * U * f["out"].abs())).sum(3, keepdim=True)
        rest = 0 * rest
    ds = w * (dp - delta) * cfg.scale
    eds = cfg.scale * w * ((dp - delta).abs() * (share + 4 * U + f["split"]) + edp + edelta)
    n = f["hit"].sum(3, keepdim=True)
    dq = ds @ f["k"]
    eq = (eds + n * U * ds.abs() + cfg.scale * 2.0 ** -9 * rest * w) @ f["k"].abs()
    fold = lambda t: t.reshape(B, cfg.heads_kv, G, *t.shape[2:]).sum(2)  # noqa: E731
    rows = (G * f["hit"].sum(2))[..., None]  # terms of a key's sums
    dk = fold(ds.transpose(2, 3) @ f["q"])
    ek = fold((eds.transpose(2, 3) + rows * U * ds.abs().transpose(2, 3)) @ f["q"].abs())
    dv = fold(w.transpose(2, 3) @ do)
    ev = fold((w * (share + f["split"])).transpose(2, 3) @ do.abs() + rows * U * (w.transpose(2, 3) @ do.abs()))
    val, err = {"dq": dq, "dk": dk, "dv": dv}, {"dq": eq, "dk": ek, "dv": ev}
    return ({x: _heads(t) for x, t in val.items()},
            {x: _heads(err[x] + h * (val[x].abs() + err[x])) for x in val})


def slot(p, S, n_sink):
    return p if p < S else n_sink + (p - n_sink) % (S - n_sink)
