"""Layer norm in 64 bits, and bounds on what a 32-bit evaluation of it may be off.

Bounds.  With u = 2^-24: a sum over a row is formed by lanes of at most 32 elements
each and at most 17 additions between them, so it is off by at most 60 u of the sum
of absolute values, and with the roundings of its terms by 64 u.  The mean is a sum
in 64 bits, rounded once; 64 u of the mean absolute deviation is allowed beside that
rounding.  A deviation is rounded twice (2 u).  The variance is off by 2 * 64 u and
4 u of itself at most, its root by half of that and 2 u, and what a deviation is off
by counts once more.  K = 96 covers each factor.
Storing adds half a step of the storage type.  A sum over n rows: n / 1024 rows a
lane, 16 lanes and 1024 / 16 + 16 parts in order: (100 + n / 1024) u and 4 u of the
products."""
import torch

U = 2.0 ** -24
K = 96
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step, relative


def forward(x, weight, bias, eps, dtype):
    """x [B, L, D] in 64 bits -> ({"y", "mean", "rstd"}, their bounds)"""
    w = torch.ones(x.shape[2], dtype=torch.float64) if weight is None else weight
    b = torch.zeros(x.shape[2], dtype=torch.float64) if bias is None else bias
    mean = x.mean(2)
    d = x - mean[..., None]
    rstd = (d.square().mean(2) + eps).rsqrt()
    xh = d * rstd[..., None]
    y = xh * w + b
    spread = d.abs().mean(2)
    ey = K * U * w.abs() * (xh.abs() + (spread * rstd)[..., None]) + 4 * U * (y.abs() + b.abs())
    return ({"y": y, "mean": mean, "rstd": rstd},
            {"y": ey + HALF[dtype] * (y.abs() + ey), "mean": U * mean.abs() + K * U * spread, "rstd": K * U * rstd})


def backward(x, dy, mean, rstd, weight, dtype):
    """mean and rstd as the forward stored them."""
    w = torch.ones(x.shape[2], dtype=torch.float64) if weight is None else weight
    xh = (x - mean[..., None]) * rstd[..., None]
    g = dy * w
    c1, c2 = g.mean(2, keepdim=True), (g * xh).mean(2, keepdim=True)
    r = rstd[..., None]
    dx = r * (g - c1 - xh * c2)
    edx = K * U * r * (g.abs() + g.abs().mean(2, keepdim=True) + xh.abs() * (g * xh).abs().mean(2, keepdim=True))
    n = 104 + x.shape[0] * x.shape[1] / 1024
    return ({"dx": dx, "dweight": (dy * xh).sum((0, 1)), "dbias": dy.sum((0, 1))},
            {"dx": edx + HALF[dtype] * (dx.abs() + edx), "dweight": n * U * (dy * xh).abs().sum((0, 1)),
             "dbias": n * U * dy.abs().sum((0, 1))})
