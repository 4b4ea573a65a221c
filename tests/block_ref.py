"""Block selection and the attention over selected blocks in 64 bits, and bounds
on what a computation with 32-bit sums may be off.

Bounds.  u = 2^-24; h is half a step of the storage type, 2^-8 for bf16.
A score (a sum of d_k products, scaled) is off by at most
D = (d_k + 4) u scale sum |q k| + 4 u |s|, the largest of which in a row, twice
(numerator and normaliser), is the relative error of a softmax weight, with
(n + 32) u for the exponential and the sum over n keys.  For bf16 each weight
is rounded once more for its product: h.  An output is off by that share of
sum p |v| and by half a step of itself.
Gradients: dp (a sum of d_v products) is off by (d_v + 4) u sum |do v|, delta
likewise and, as it is formed from the stored output, by h sum |do o|; the score's
gradient p (dp - delta) scale adds the weight's share and, for bf16, its
rounding h; the sums over keys or rows add (number of terms) u."""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def positions(B, L, S, start=None, lens=None):
    """[B, L], -1 for padding."""
    p = (np.zeros(B, np.int64) if start is None else np.asarray(start, np.int64))[:, None] + np.arange(L)
    n = np.full(B, S) if lens is None else np.minimum(lens, S)
    return np.where((p >= 0) & (p < n[:, None]), p, -1)


def means(k, block, lens=None):
    B, S, H, d = k.shape
    out = np.zeros((B, H, -(-S // block), d))
    for b in range(B):
        w = max(0, min(S if lens is None else int(lens[b]), S)) // block
        out[b, :, :w] = k[b, :w * block].reshape(w, block, H, d).mean(1).swapaxes(0, 1)
    return out


def select(q, c, cfg, S, start=None, lens=None):
    """Row by row: the forced blocks, then the others by score, a lower index first among equals."""
    B, L, hq, _ = q.shape
    H = c.shape[1]
    sel = np.full((B, H, L, cfg.n_select), -1, np.int32)
    p = positions(B, L, S, start, lens)
    for b, h, i in np.ndindex(B, H, L):
        if p[b, i] < 0:
            continue
        own = p[b, i] // cfg.block
        forced = sorted({j for j in range(min(cfg.n_first, own + 1))} | set(range(max(0, own - cfg.n_recent + 1), own + 1)))
        score = c[b, h] @ q[b, i, h * (hq // H):(h + 1) * (hq // H)].sum(0)
        rest = sorted((j for j in range(own + 1) if j not in forced), key=lambda j: (-score[j], j))
        chosen = sorted(forced + rest[:cfg.n_select - len(forced)])
        sel[b, h, i, :len(chosen)] = chosen
    return sel


def allowed(sel, cfg, p, S):
    """[B, H, L, S] from any contents of sel, by the documented rule."""
    B, H, L, n = sel.shape
    hit = np.zeros((B, H, L, S), bool)
    for b, h, i in np.ndindex(B, H, L):
        last = -1
        if p[b, i] < 0:
            continue
        for j in sel[b, h, i]:
            if last < j <= p[b, i] // cfg.block:
                last = int(j)
                hit[b, h, i, last * cfg.block:min((last + 1) * cfg.block, p[b, i] + 1)] = True
    return hit


def _heads(t):
    return t.transpose(0, 2, 1, 3)


def forward(q, k, v, sel, cfg, start=None, lens=None):
    """(values, bounds), each {"out", "lse"}, and what the gradients need."""
    B, L, S, G, h = q.shape[0], q.shape[1], k.shape[1], cfg.heads_q // cfg.heads_kv, HALF[cfg.dtype]
    p = positions(B, L, S, start, lens)
    hit = np.repeat(allowed(sel, cfg, p, S), G, axis=1)
    kk, vv, qq = np.repeat(_heads(k), G, axis=1), np.repeat(_heads(v), G, axis=1), _heads(q)
    kk, vv = np.nan_to_num(kk), np.nan_to_num(vv)  # what lies behind the sequences may be anything
    s = qq @ kk.swapaxes(2, 3) * cfg.scale
    size = np.abs(qq) @ np.abs(kk).swapaxes(2, 3) * cfg.scale
    some = hit.any(3, keepdims=True)
    top = np.where(some, np.where(hit, s, -np.inf).max(3, keepdims=True), 0)
    e = np.where(hit, np.exp(np.where(hit, s - top, 0)), 0)
    total = e.sum(3, keepdims=True)
    w = e / np.where(some, total, 1)
    off = (np.where(hit, (cfg.d_k + 4) * U * size + 4 * U * np.abs(s), 0)).max(3, keepdims=True)
    share = 2 * off + (hit.sum(3, keepdims=True) + 32) * U
    out = w @ vv
    rounded = h if cfg.dtype == "bf16" else 0.0
    eo = (share + rounded) * (w @ np.abs(vv))
    with np.errstate(all="ignore"):
        lse = np.where(some, top + np.log(total), -np.inf)[..., 0]
    el = np.where(some, share + 4 * U * np.abs(np.where(some, lse[..., None], 0)), 0)[..., 0]
    keep = {"w": w, "hit": hit, "share": share, "q": qq, "k": kk, "v": vv, "out": out}
    return ({"out": _heads(out), "lse": lse}, {"out": _heads(eo + h * (np.abs(out) + eo)), "lse": el}, keep)


def backward(q, k, v, sel, dout, cfg, start=None, lens=None):
    _, _, f = forward(q, k, v, sel, cfg, start, lens)
    B, L, S, G, h = q.shape[0], q.shape[1], k.shape[1], cfg.heads_q // cfg.heads_kv, HALF[cfg.dtype]
    rounded = h if cfg.dtype == "bf16" else 0.0
    w, do = f["w"], _heads(dout)
    live = (positions(B, L, S, start, lens) >= 0)[:, None, :, None]
    do = np.where(live, do, 0)
    dp = do @ f["v"].swapaxes(2, 3)
    edp = (cfg.d_v + 4) * U * (np.abs(do) @ np.abs(f["v"]).swapaxes(2, 3))
    delta = (do * f["out"]).sum(3, keepdims=True)
    edelta = (h + (cfg.d_v + 4) * U) * np.abs(do * f["out"]).sum(3, keepdims=True)
    ds = w * (dp - delta) * cfg.scale
    eds = cfg.scale * w * (np.abs(dp - delta) * (f["share"] + 4 * U + rounded) + edp + edelta)
    n = f["hit"].sum(3, keepdims=True)
    dq = ds @ f["k"]
    eq = (eds + n * U * np.abs(ds)) @ np.abs(f["k"])
    fold = lambda t: t.reshape(B, cfg.heads_kv, G, *t.shape[2:]).sum(2)  # noqa: E731
    rows = np.repeat(fold(f["hit"].sum(2)[..., None]), G, axis=1)  # terms of a key's sums
    dk = fold(ds.swapaxes(2, 3) @ f["q"])
    ek = fold((eds.swapaxes(2, 3) + rows * U * np.abs(ds).swapaxes(2, 3)) @ np.abs(f["q"]))
    dv = fold(w.swapaxes(2, 3) @ do)
    ev = fold((w * (f["share"] + rounded)).swapaxes(2, 3) @ np.abs(do) + rows * U * (w.swapaxes(2, 3) @ np.abs(do)))
    val = {"dq": _heads(dq), "dk": _heads(dk), "dv": _heads(dv)}
    err = {"dq": _heads(eq), "dk": _heads(ek), "dv": _heads(ev)}
    return val, {x: err[x] + h * (np.abs(val[x]) + err[x]) for x in val}
