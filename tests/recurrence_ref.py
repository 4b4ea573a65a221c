"""The gated linear recurrence in 64 bits, position by position, and bounds on
what a 32-bit evaluation of it may be off.

Bounds.  With u = 2^-24 a computed decay, input scale or slope is off by at
most K u of itself, K = 16 + 2 |z + b| + 12 |log alpha|: the rounding of z + b
moves log alpha by at most u |z + b| of its own, the exponential and the
logarithm's series take a few u each, and the exponential returns an absolute
error of its argument (log alpha, known to 10 u of itself) as a relative one.
An error then runs through the recurrence like the state itself:
    E_t = alpha_t E_{t-1} + (K_t + 4) u (alpha_t M_{t-1} + |beta_t x_t|),
with M the recurrence over absolute values, where the 4 stands for the
roundings of one step and of one factor of a chunk's decay product.
Storing adds half a step of the storage type."""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step, relative


def gates(z, bias, gamma, mode):
    zb = z + bias
    la = (np.minimum(zb, 0) - np.log1p(np.exp(-np.abs(zb)))) / gamma
    alpha = np.exp(la)
    with np.errstate(all="ignore"):
        beta, slope = {
            "plain": lambda: (np.ones_like(la), np.zeros_like(la)),
            "convex": lambda: (-np.expm1(la), -alpha),
            "norm": lambda: (np.sqrt(-np.expm1(2 * la)), -alpha ** 2 / np.sqrt(-np.expm1(2 * la))),
        }[mode]()
        sig = 1 / (1 + np.exp(zb))
    K = 16 + 2 * np.abs(zb) + 12 * np.abs(la)
    return alpha, beta, slope, sig, K


def forward(x, z, bias, gamma, mode, mask=None, h_in=None, dtype="f32"):
    """{"y", "h_out"} and {"y", "h_out"} bounds."""
    B, L, D = x.shape
    alpha, beta, _, _, K = gates(z, bias, gamma, mode)
    on = np.ones((B, L, 1), bool) if mask is None else (mask != 0)[:, :, None]
    h = np.zeros((B, D)) if h_in is None else h_in.copy()
    M, E = np.abs(h), np.zeros((B, D))
    y, ey = np.zeros_like(x), np.zeros_like(x)
    for t in range(L):
        a, ux = alpha[:, t], np.where(on[:, t], beta[:, t] * x[:, t], 0)
        o = on[:, t]
        E = np.where(o, a * E + (K[:, t] + 4) * U * (a * M + np.abs(ux)), E)
        M = np.where(o, a * M + np.abs(ux), M)
        h = np.where(o, a * h + ux, h)
        y[:, t], ey[:, t] = np.where(o, h, 0), np.where(o, E, 0)
    return {"y": y, "h_out": h}, {"y": ey + HALF[dtype] * (np.abs(y) + ey), "h_out": E + U * np.abs(h)}


def backward(x, z, dy, bias, gamma, mode, mask=None, h_in=None, dh_out=None, dtype="f32"):
    B, L, D = x.shape
    alpha, beta, slope, sig, K = gates(z, bias, gamma, mode)
    on = np.ones((B, L, 1), bool) if mask is None else (mask != 0)[:, :, None]
    h = np.zeros((B, D)) if h_in is None else h_in.copy()
    M, E = np.abs(h), np.zeros((B, D))
    hb, eb = np.zeros_like(x), np.zeros_like(x)
    for t in range(L):
        hb[:, t], eb[:, t] = h, E
        o, a, ux = on[:, t], alpha[:, t], np.where(on[:, t], beta[:, t] * x[:, t], 0)
        E = np.where(o, a * E + (K[:, t] + 4) * U * (a * M + np.abs(ux)), E)
        M = np.where(o, a * M + np.abs(ux), M)
        h = np.where(o, a * h + ux, h)
    c = np.zeros((B, D)) if dh_out is None else dh_out.copy()
    M, E = np.abs(c), np.zeros((B, D))
    dx, dz, ex, ez = (np.zeros_like(x) for _ in range(4))
    for t in reversed(range(L)):
        o, a = on[:, t], alpha[:, t]
        d = np.where(o, dy[:, t], 0) if dy is not None else np.zeros((B, D))
        dh, mh, eh = c + d, M + np.abs(d), E + 2 * U * (M + np.abs(d))
        with np.errstate(all="ignore"):
            inner = a * hb[:, t] + slope[:, t] * x[:, t]
            mag = np.abs(a * hb[:, t]) + np.abs(slope[:, t] * x[:, t])
            s = sig[:, t] / gamma
            dx[:, t] = np.where(o, beta[:, t] * dh, 0)
            ex[:, t] = np.where(o, np.abs(beta[:, t]) * eh + (K[:, t] + 2) * U * np.abs(beta[:, t] * dh), 0)
            dz[:, t] = np.where(o, dh * inner * s, 0)
            ez[:, t] = np.where(o, s * (eh * mag + np.abs(dh) * (a * eb[:, t] + (4 * K[:, t] + 8) * U * mag)), 0)
        E = np.where(o, a * eh + (K[:, t] + 4) * U * a * mh, eh)
        M = np.where(o, a * mh, mh)
        c = np.where(o, a * dh, dh)
    half = HALF[dtype]
    # a chunk's partial of dbias adds 64 rounded terms in 32 bits; the partials meet in 64 bits
    return ({"dx": dx, "dz": dz, "dbias": dz.sum((0, 1)), "dh_in": c},
            {"dx": ex + half * (np.abs(dx) + ex), "dz": ez + half * (np.abs(dz) + ez),
             "dbias": (ez + 66 * U * np.abs(dz)).sum((0, 1)) + U * np.abs(dz.sum((0, 1))), "dh_in": E + U * np.abs(c)})
