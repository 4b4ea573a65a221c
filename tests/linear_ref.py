"""Linear attention with a decay per head in 64 bits, position by position, and
bounds on what an evaluation in chunks of 64 with 32-bit sums may be off.

Bounds.  With u = 2^-24, per position and with all products over absolute values:
a weight gamma^n is off by at most 3 n |log gamma| u and 2 u of itself (its exponent
is a rounded product, and the exponential returns an absolute error of its argument
as a relative one); a chunk's sum of 64 products by 64 u; with bf16 inputs a weighted
value that enters a product as two bf16 values by 2^-18 = 64 u (each rounding leaves
2^-9 of what it rounds).  So the state's error runs with it:
    E_t = gamma (E_{t-1} + (3 |log gamma| + 2) u M_{t-1}) + KS u |k_t| |v_t|,
with M the state over absolute values and KS = 136.  The product with q sums d_k terms
in either part, of which one enters rounded and the other has 64 weights, which are sums
of d_k products: KQ = d_k + 144 (2 * 64 and the products' own roundings).  Storing adds
half a step of the storage type.  The gradients are the same recurrence with other
operands."""
import torch

U = 2.0 ** -24
KS = 136
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def walk(q, k, v, log_decay, lens, state, scale, dtype, lead=0):
    """q, k [B, L, H, dk], v [B, L, H, dv] in 64 bits and in the order of the walk, log_decay [H], lens [B] list, state
    [B, H, dk, dv] or None -> ((out, last state), (their bounds)).  lead: the first step does not decay the state."""
    B, L, H, dk = q.shape
    lg = log_decay.clamp(min=-1e30)
    gamma = lg.exp()[:, None, None]
    rate = (3 * lg.abs().clamp(max=200) + 2)[:, None, None] * U  # gamma^n is 0 in fp32 long before n |log gamma| = 200
    S = torch.zeros((B, H, dk, v.shape[3]), dtype=torch.float64) if state is None else state.clone()
    M, E = S.abs(), 2 * U * S.abs()
    n = torch.tensor(lens)[:, None, None, None]
    out, eo = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(L):
        kv = k[:, t, :, :, None] * v[:, t, :, None]
        g = torch.ones_like(gamma) if lead and t == 0 else gamma
        on = t < n
        E = torch.where(on, g * (E + rate * M) + KS * U * kv.abs(), E)
        M = torch.where(on, g * M + kv.abs(), M)
        S = torch.where(on, g * S + kv, S)
        out[:, t] = scale * (q[:, t, :, None] @ S)[:, :, 0]
        eo[:, t] = scale * (q[:, t, :, None].abs() @ (E + (dk + 144) * U * M))[:, :, 0]
    here = torch.arange(L)[None, :, None, None] < n
    out, eo = torch.where(here, out, 0.0), torch.where(here, eo, 0.0)
    return (out, S), (eo + HALF[dtype] * (out.abs() + eo), E + 2 * U * S.abs())


def _turn(t, lens):
    out = t.clone()
    for b, n in enumerate(lens):
        out[b, :n] = t[b, :n].flip(0)
    return out


def backward(q, k, v, log_decay, lens, state, dout, dstate, scale, dtype):
    """{"dq", "dk", "dv", "dstate"} and their bounds."""
    (dq, _), (edq, _) = walk(dout, v, k, log_decay, lens, None if state is None else state.transpose(2, 3), scale, dtype)
    qt, kt, vt, dt = (_turn(t, lens) for t in (q, k, v, dout))
    first = None if dstate is None else dstate / scale
    (dk, _), (edk, _) = walk(vt, dt, qt, log_decay, lens, None if first is None else first.transpose(2, 3), scale, dtype, 1)
    (dv, last), (edv, el) = walk(kt, qt, dt, log_decay, lens, first, scale, dtype, 1)
    lg = log_decay.clamp(min=-1e30)
    g = torch.where(torch.tensor(lens)[:, None, None, None] > 0, scale * lg.exp()[:, None, None], scale)
    more = (3 * lg.abs().clamp(max=200) + 6)[:, None, None] * U  # the last decay, and both factors of scale
    return ({"dq": dq, "dk": _turn(dk, lens), "dv": _turn(dv, lens), "dstate": g * last},
            {"dq": edq, "dk": _turn(edk, lens), "dv": _turn(edv, lens), "dstate": g * (el + more * last.abs())})
