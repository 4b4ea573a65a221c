"""Cases, plain forms and exact values of the operators that stand with the MS-GLA layer in one stack.

Three operators, measured alone and as a user's program calls them:

* layer norm over the channels of every position, forward and backward: what stands before each mixer;
* linear attention with a decay for each head,  S_t = gamma_h S_{t-1} + k_t^T v_t,  o_t = scale q_t S_t:
  forward over a sequence, backward, one streaming step;
* attention with a sliding window and a few first tokens that stay visible: a query at position p attends
  the keys j <= p with j > p - window or j < n_sink: forward, backward, and one streaming step that puts a
  token's key and value into a rolling cache and attends.

`own` chooses between the plain form (elementary torch operations) and the framework's
kernels; `exact` gives the same values in 64 bits, written apart from both.
"""
import math

import torch

own = False

CHUNK = 64  # positions that the plain form of linear attention takes at once


# ---- cases --------------------------------------------------------------------

def _norm(name, kind, B, L, D, dtype):
    c = {"kind": kind, "B": B, "L": L, "D": D, "dtype": dtype}
    return {"name": name, **c} if name else c


def _lin(name, kind, B, L, heads, dk, dv, dtype, state=False, ragged=False):
    c = {"kind": kind, "B": B, "L": L, "heads": heads, "d_k": dk, "d_v": dv, "dtype": dtype, "state": state,
         "ragged": ragged}
    return {"name": name, **c} if name else c


def _win(name, kind, B, L, hq, hkv, dk, dv, window, n_sink, dtype, ragged=False):
    """L: the sequence's length; for a step the number of tokens that the longest sequence has had."""
    c = {"kind": kind, "B": B, "L": L, "heads_q": hq, "heads_kv": hkv, "d_k": dk, "d_v": dv, "window": window,
         "n_sink": n_sink, "dtype": dtype, "ragged": ragged}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of each of 16 streams of the layer's width: a launch's latency
        _norm("norm B16 L1 D1024", "norm_forward", 16, 1, 1024, "bf16"),
        # the training step of the layer's main batch
        _norm("norm grad B8 L2048 D1024", "norm_backward", 8, 2048, 1024, "bf16"),
        # an odd width and length in full precision
        _norm("norm grad f32 B3 L4093 D1001", "norm_backward", 3, 4093, 1001, "f32"),
        # the layer's main batch and head widths
        _lin("linear B8 L2048 H4", "lin_forward", 8, 2048, 4, 128, 256, "bf16"),
        # a long document in one sequence, continued from a state
        _lin("linear B1 L16384 H4", "lin_forward", 1, 16384, 4, 128, 256, "bf16", state=True),
        # the main batch's other half of a training step
        _lin("linear grad B8 L2048 H4", "lin_backward", 8, 2048, 4, 128, 256, "bf16"),
        # serving: one token of each of 16 sequences
        _lin("linear step B16 H4", "lin_step", 16, 1, 4, 128, 256, "bf16", state=True),
        # the main batch, grouped heads
        _win("window B8 L2048 H16/4 W512", "win_forward", 8, 2048, 16, 4, 128, 128, 512, 4, "bf16"),
        # a long prefill with the layer's own head widths
        _win("window B1 L16384 H8/2 dv256 W4096", "win_forward", 1, 16384, 8, 2, 128, 256, 4096, 64, "bf16"),
        # training on longer sequences
        _win("window grad B2 L4096 H16/4 W1024", "win_backward", 2, 4096, 16, 4, 128, 128, 1024, 4, "bf16"),
        # a short padded batch in full precision with groups of three and odd lengths
        _win("window grad f32 B3 L999 H6/2 padded", "win_backward", 3, 999, 6, 2, 64, 96, 100, 3, "f32", ragged=True),
        # serving: one token of each of 16 sequences over rolling caches, most of them turned over
        _win("window step B16 H16/4 W4096", "win_step", 16, 20000, 16, 4, 128, 128, 4096, 4, "bf16", ragged=True),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    what = rng.choice(("norm", "linear", "linear", "window", "window"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if what == "norm":
        D = _log_between(rng, 64, 8192)
        D = D if rng.random() < 0.4 else max(64, D // 64 * 64)
        rows = _log_between(rng, 1, max(2, 33554432 // D))
        B = min(rows, _log_between(rng, 1, 16))
        return _norm("", rng.choice(("norm_forward", "norm_backward")), B, max(1, rows // B), D, dtype)
    if what == "linear":
        kind = rng.choice(("lin_forward", "lin_backward", "lin_step"))
        heads = rng.choice((1, 2, 3, 4, 8, 16))
        dk, dv = rng.choice((32, 64, 80, 128, 256)), rng.choice((64, 96, 128, 256))
        if kind == "lin_step":
            return _lin("", kind, _log_between(rng, 1, 128), 1, heads, dk, dv, dtype, state=True)
        B = _log_between(rng, 1, 16)
        L = _log_between(rng, 33, max(64, min(16384, 131072 // (B * heads))))
        return _lin("", kind, B, L, heads, dk, dv, dtype, rng.random() < 0.5, rng.random() < 0.4)
    kind = rng.choice(("win_forward", "win_forward", "win_backward", "win_step"))
    hkv = rng.choice((1, 2, 4))
    hq = hkv * rng.choice((1, 2, 3, 4, 5, 8, 16))
    dk, dv = rng.choice((32, 64, 80, 128)), rng.choice((64, 96, 128, 256))
    window, n_sink = _log_between(rng, 16, 4096), rng.choice((0, 1, 4, 4, 16, 64, 100))
    if kind == "win_step":
        return _win("", kind, _log_between(rng, 1, 32), _log_between(rng, 20, 30000), hq, hkv, dk, dv, window, n_sink,
                    dtype, True)
    B = rng.choice((1, 2, 3, 4))
    top = int(math.sqrt(2.0e9 / (B * hq * (2 if kind == "win_backward" else 1))))
    return _win("", kind, B, _log_between(rng, 100, max(200, min(8192, top))), hq, hkv, dk, dv, window, n_sink, dtype,
                rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """Tokens of each sequence: all of them, or from the whole length down to a third of it."""
    B, L = case["B"], case["L"]
    return [max(1, L - (b * 2 * L) // (3 * B)) if case.get("ragged") else L for b in range(B)]


def _slots(case):
    """Positions that a rolling cache holds: the first tokens, the window, and some room."""
    return case["n_sink"] + case["window"] + case["window"] // 8


def _slot(case, p):
    """Where a rolling cache keeps a position."""
    ns, S = case["n_sink"], _slots(case)
    return torch.where(p < ns, p, ns + (p - ns) % (S - ns))


def _slow(g, B, L, H, d, every, share):
    """Vectors whose topic changes every few positions, as the queries and keys of a text do."""
    r = lambda n: torch.randn((B, n, H, d), generator=g, device="cuda")  # noqa: E731
    topic = r((L + every - 1) // every).repeat_interleave(every, dim=1)[:, :L]
    return topic * share + r(L) * math.sqrt(1 - share * share)


def _plan(case):
    """The framework's handle of an operator."""
    from scale_gla_layer_amd import config, runner
    if case["kind"].startswith("norm"):
        return runner.DeviceLayerNorm(config.LayerNormConfig(case["D"], dtype=case["dtype"]))
    if case["kind"].startswith("lin"):
        return runner.DeviceLinearAttention(config.LinearAttentionConfig(case["heads"], case["d_k"], case["d_v"],
                                                                         dtype=case["dtype"]))
    return runner.DeviceWindowAttention(config.WindowAttentionConfig(
        case["heads_q"], case["heads_kv"], case["d_k"], case["d_v"], case["window"], case["n_sink"],
        dtype=case["dtype"]))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, L, kind = _type(case), case["B"], case["L"], case["kind"]
    s = {"case": case, "plan": _plan(case) if own else None}
    r = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    if kind.startswith("norm"):
        D = case["D"]
        # a residual stream: channels of several sizes, some with a mean of their own
        s["x"] = (r(B, L, D) * (0.5 + 2 * torch.rand(D, generator=g, device="cuda")) + 0.7 * r(D)).to(dt)
        s["weight"], s["bias"] = 1 + 0.3 * r(D), 0.3 * r(D)
        if kind == "norm_backward":
            s["dy"] = r(B, L, D).to(dt)
            s["mean"], s["rstd"] = _statistics(s["x"])
        return s
    if kind.startswith("lin"):
        H, dk, dv = case["heads"], case["d_k"], case["d_v"]
        s["q"], s["k"], s["v"] = r(B, L, H, dk).to(dt), r(B, L, H, dk).to(dt), r(B, L, H, dv).to(dt)
        # decays from about eight positions to about a thousand, as heads of several ranges have them
        reach = torch.arange(H, device="cuda") * (6 / max(1, H - 1)) + 3 + torch.rand(H, generator=g, device="cuda")
        s["log_decay"] = torch.log1p(-torch.exp2(-reach))
        s["lens"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32) if case["ragged"] else None
        s["state"] = 3 * r(B, H, dk, dv) if case["state"] else None
        if kind == "lin_backward":
            s["dout"] = r(B, L, H, dv).to(dt)
            s["dstate"] = r(B, H, dk, dv) if case["state"] else None
        if kind == "lin_step":
            s["q"], s["k"], s["v"] = s["q"][:, 0], s["k"][:, 0], s["v"][:, 0]
            s["state_out"] = torch.empty_like(s["state"])
        return s
    hq, hkv, dk, dv = case["heads_q"], case["heads_kv"], case["d_k"], case["d_v"]
    if kind == "win_step":
        S = _slots(case)
        s["q"], s["kt"], s["vt"] = r(B, hq, dk).to(dt), r(B, hkv, dk).to(dt), r(B, hkv, dv).to(dt)
        s["k"], s["v"] = _slow(g, B, S, hkv, dk, 64, 0.6).to(dt), r(B, S, hkv, dv).to(dt)
        s["pos"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32) - 1
        return s
    s["k"], s["v"] = _slow(g, B, L, hkv, dk, 64, 0.6).to(dt), r(B, L, hkv, dv).to(dt)
    s["lens"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32) if case["ragged"] else None
    # queries of neighbouring positions, and of the heads of a group, look for similar things
    q = _slow(g, B, L, hkv, dk, 32, 0.6)[:, :, :, None] * 0.7 + r(B, L, hkv, hq // hkv, dk) * 0.7
    s["q"] = q.reshape(B, L, hq, dk).to(dt)
    if kind == "win_backward":
        s["out"], s["lse"] = _attend(case, s["q"], s["k"], s["v"], s["lens"])
        s["dout"] = r(B, L, hq, dv).to(dt)
    return s


# ---- plain forms --------------------------------------------------------------

EPS = 1e-5


def _statistics(x):
    x = x.float()
    mean = x.mean(2, keepdim=True)
    var = (x - mean).square().mean(2)
    return mean[:, :, 0], torch.rsqrt(var + EPS)


def _layer_norm(case, s):
    x = s["x"].float()
    if case["kind"] == "norm_forward":
        mean, rstd = _statistics(s["x"])
        y = (x - mean[:, :, None]) * rstd[:, :, None] * s["weight"] + s["bias"]
        return {"y": y.to(_type(case)), "mean": mean, "rstd": rstd}
    xh = (x - s["mean"][:, :, None]) * s["rstd"][:, :, None]
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = (g - g.mean(2, keepdim=True) - xh * (g * xh).mean(2, keepdim=True)) * s["rstd"][:, :, None]
    return {"dx": dx.to(_type(case)), "dweight": (dy * xh).sum((0, 1), dtype=torch.float64).float(),
            "dbias": dy.sum((0, 1), dtype=torch.float64).float()}


def _linear(q, k, v, rate, state, lens):
    """o_t = q_t S_t and the state after the last token, for S_t = gamma S_{t-1} + k_t^T v_t, in chunks: q, k
    [B, L, H, dk], v [B, L, H, dv] with zeroes behind a sequence's end, rate [H] = log gamma in 64 bits, state
    [B, H, dk, dv] or None, lens [B]."""
    B, L, H, _ = q.shape
    C, n, dev = CHUNK, -(-L // CHUNK), q.device
    q, k, v = (torch.cat((t, t.new_zeros((B, n * C - L, *t.shape[2:]))), 1).transpose(1, 2).unflatten(2, (n, C))
               for t in (q, k, v))
    i, m = torch.arange(C, device=dev), torch.arange(n + 1, device=dev)
    until = torch.minimum(lens[:, None], m * C)  # tokens before each chunk, and all of them
    here = until[:, 1:] - until[:, :-1]

    def power(e):  # gamma^e [.., H, ..] of whole numbers [.., 1, ..], 0 where e is negative
        r = rate.reshape(-1, *[1] * (e.dim() - 2))
        return torch.where(e >= 0, torch.exp(r * e.clamp(min=0)), 0.0).float()

    within = power((i[:, None] - i)[None, None, None])[0]  # [H, 1, C, C]
    out = ((q @ k.transpose(3, 4)) * within) @ v
    left = power((here[:, :, None] - 1 - i)[:, None])  # [B, H, n, C]: until the end of the chunk
    grown = (k * left[..., None]).transpose(3, 4) @ v  # what each chunk adds to the state
    gap = torch.where(m[:, None] > m[:n], until[:, :, None] - until[:, None, 1:], -1)
    states = (power(gap[:, None]) @ grown.flatten(3)).unflatten(3, grown.shape[3:])  # before each chunk, and the last
    if state is not None:
        states = states + power(until[:, None])[..., None, None] * state[:, :, None]
    out = out + (q * power((i + 1)[None, None])[0][:, None, :, None]) @ states[:, :, :n]
    return out.flatten(2, 3)[:, :, :L].transpose(1, 2), states[:, :, n]


def _linear_attention(case, s):
    dt, scale, rate = _type(case), case["d_k"] ** -0.5, s["log_decay"].double()
    if case["kind"] == "lin_step":
        q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
        S = torch.exp(rate).float()[:, None, None] * s["state"] + k[:, :, :, None] * v[:, :, None]
        return {"out": (scale * (q[:, :, None] @ S)[:, :, 0]).to(dt), "state": S}
    B, L, dev = case["B"], case["L"], s["q"].device
    lens = torch.full((B,), L, device=dev) if s["lens"] is None else s["lens"].long()
    at = torch.arange(L, device=dev)
    token = (at < lens[:, None])[:, :, None, None]
    real = lambda t: torch.where(token, t.float(), 0.0)  # noqa: E731
    q, k, v = real(s["q"]), real(s["k"]), real(s["v"])
    if case["kind"] == "lin_forward":
        out, state = _linear(q, k, v, rate, s["state"], lens)
        return {"out": (out * scale).to(dt), "state": state}
    # each gradient is linear attention itself: dq of (do, v, k); from the last token on dk of (v, do, q) and
    # dv of (k, q, do), whose state before the first step is dstate
    do = real(s["dout"])
    dq, _ = _linear(do, v, k, rate, None if s["state"] is None else s["state"].transpose(2, 3), lens)
    order = ((lens[:, None] - 1 - at) % L)[:, :, None, None]
    turn = lambda t: torch.where(token, t.gather(1, order.expand(t.shape)), 0.0)  # noqa: E731
    gamma = torch.exp(rate)[:, None, None]
    entry = None if s["dstate"] is None else (s["dstate"] / gamma / scale).float()
    dk, _ = _linear(turn(v), turn(do), turn(q), rate, None if entry is None else entry.transpose(2, 3), lens)
    dv, first = _linear(turn(k), turn(q), turn(do), rate, entry, lens)
    out = {"dq": (dq * scale).to(dt), "dk": (turn(dk) * scale).to(dt), "dv": (turn(dv) * scale).to(dt)}
    return out if s["state"] is None else {**out, "dstate": (first * gamma * scale).float()}


def _allowed(case, L, lens, device):
    """Whether the query at a position attends a key: [B or 1, 1, 1, L, L]."""
    key, p = torch.arange(L, device=device), torch.arange(L, device=device)[:, None]
    hit = ((key <= p) & ((key > p - case["window"]) | (key < case["n_sink"])))[None]
    if lens is not None:
        hit = hit & (p < lens[:, None, None])
    return hit[:, None, None]


def _grouped(t, H):
    """[B, L, H G, d] as [B, H, G, L, d] in 32 bits."""
    B, L, hq, d = t.shape
    return t.float().reshape(B, L, H, hq // H, d).permute(0, 2, 3, 1, 4).contiguous()


def _flat(t, dt):
    B, H, G, L, d = t.shape
    return t.permute(0, 3, 1, 2, 4).reshape(B, L, H * G, d).to(dt)


def _weights(case, q, k, lens):
    hit = _allowed(case, q.shape[3], lens, q.device)
    score = torch.where(hit, q @ k.transpose(3, 4) / math.sqrt(case["d_k"]), -math.inf)
    top = score.amax(4, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(4, keepdim=True)
    return p / torch.where(total > 0, total, 1.0), (top + torch.log(total)).squeeze(4)


def _attend(case, q, k, v, lens):
    H, dt = case["heads_kv"], q.dtype
    p, lse = _weights(case, _grouped(q, H), _grouped(k, H), lens)
    return _flat(p @ _grouped(v, H), dt), lse.flatten(1, 2)


def _attend_back(case, s):
    H, dt = case["heads_kv"], _type(case)
    q, k, v, do = (_grouped(s[n], H) for n in ("q", "k", "v", "dout"))
    p, _ = _weights(case, q, k, s["lens"])
    dp = do @ v.transpose(3, 4)
    ds = p * (dp - (p * dp).sum(4, keepdim=True)) / math.sqrt(case["d_k"])
    dk = (ds.transpose(3, 4) @ q).sum(2, keepdim=True)
    dv = (p.transpose(3, 4) @ do).sum(2, keepdim=True)
    return {"dq": _flat(ds @ k, dt), "dk": _flat(dk, dt), "dv": _flat(dv, dt)}


def _attend_step(case, s):
    """Puts each sequence's token into its slot and attends the window and the first tokens."""
    k, v, pos, H, ns, W = s["k"], s["v"], s["pos"].long(), case["heads_kv"], case["n_sink"], case["window"]
    B = k.shape[0]
    row = torch.arange(B, device=k.device)
    at = _slot(case, pos)
    k[row, at], v[row, at] = s["kt"], s["vt"]
    first, near = torch.arange(ns, device=k.device), torch.arange(W, device=k.device)
    key = torch.cat((first.expand(B, ns), pos[:, None] - near), 1)
    hit = torch.cat((first <= pos[:, None], (pos[:, None] - near >= ns)), 1)[:, None, None]
    slot = _slot(case, key.clamp(min=0))[:, None]
    head = torch.arange(H, device=k.device)[None, :, None]
    kk, vv = k[row[:, None, None], slot, head].float(), v[row[:, None, None], slot, head].float()
    q = s["q"].float().reshape(B, H, -1, case["d_k"])
    score = torch.where(hit, q @ kk.transpose(2, 3) / math.sqrt(case["d_k"]), -math.inf)
    p = torch.exp(score - score.amax(3, keepdim=True))
    out = (p / p.sum(3, keepdim=True)) @ vv
    return {"out": out.flatten(1, 2).to(k.dtype), "k": k, "v": v}


# ---- one pass -----------------------------------------------------------------

def _run_own(s):
    case, plan = s["case"], s["plan"]
    kind = case["kind"]
    if kind == "norm_forward":
        y, mean, rstd = plan.forward(s["x"], s["weight"], s["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_backward":
        dx, dweight, dbias = plan.backward(s["x"], s["dy"], s["mean"], s["rstd"], s["weight"], s["bias"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if kind == "lin_forward":
        out, state = plan.forward(s["q"], s["k"], s["v"], s["log_decay"], lens=s["lens"], state_in=s["state"])
        return {"out": out, "state": state}
    if kind == "lin_backward":
        dq, dk, dv, dstate = plan.backward(s["q"], s["k"], s["v"], s["log_decay"], s["dout"], lens=s["lens"],
                                           state_in=s["state"], dstate_out=s["dstate"])
        out = {"dq": dq, "dk": dk, "dv": dv}
        return {**out, "dstate": dstate} if dstate is not None else out
    if kind == "lin_step":
        out, state = plan.step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], state_out=s["state_out"])
        return {"out": out, "state": state}
    if kind == "win_forward":
        out, lse = plan.forward(s["q"], s["k"], s["v"], lens=s["lens"])
        return {"out": out, "lse": lse}
    if kind == "win_backward":
        dq, dk, dv = plan.backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], lens=s["lens"])
        return {"dq": dq, "dk": dk, "dv": dv}
    out = plan.step(s["q"], s["kt"], s["vt"], s["k"], s["v"], s["pos"])
    return {"out": out, "k": s["k"], "v": s["v"]}


def run(state):
    case, s = state["case"], state
    if own:
        return _run_own(s)
    if case["kind"].startswith("norm"):
        return _layer_norm(case, s)
    if case["kind"].startswith("lin"):
        return _linear_attention(case, s)
    if case["kind"] == "win_forward":
        out, lse = _attend(case, s["q"], s["k"], s["v"], s["lens"])
        return {"out": out, "lse": lse}
    if case["kind"] == "win_backward":
        return _attend_back(case, s)
    return _attend_step(case, s)


def work(case):
    e, B, L, kind = (2 if case["dtype"] == "bf16" else 4), case["B"], case["L"], case["kind"]
    lengths = _lengths(case)
    tokens = sum(lengths)
    if kind.startswith("norm"):
        D = case["D"]
        if kind == "norm_forward":
            return {"bytes": 2 * e * B * L * D + 8 * B * L + 8 * D, "flops": 8 * B * L * D}
        return {"bytes": 3 * e * B * L * D + 8 * B * L + 12 * D, "flops": 16 * B * L * D}
    if kind.startswith("lin"):
        H, dk, dv = case["heads"], case["d_k"], case["d_v"]
        state = 4 * B * H * dk * dv
        if kind == "lin_step":
            return {"bytes": 2 * state + 2 * e * B * H * (dk + dv), "flops": 5 * B * H * dk * dv}
        # a position's product with the state and its share of the state
        once = 4 * tokens * H * dk * dv
        if kind == "lin_forward":
            # inputs are read where there are tokens; outputs are written everywhere
            return {"bytes": e * H * (tokens * (2 * dk + dv) + B * L * dv) + state * (2 if case["state"] else 1),
                    "flops": once}
        return {"bytes": e * H * (tokens * (2 * dk + 2 * dv) + B * L * (2 * dk + dv)) + (3 * state if case["state"] else 0),
                "flops": 3 * once}
    hq, hkv, dk, dv, W, ns = (case[x] for x in ("heads_q", "heads_kv", "d_k", "d_v", "window", "n_sink"))
    if kind == "win_step":
        keys = sum(min(l, W) + min(ns, max(0, l - W)) for l in lengths)
        return {"bytes": keys * hkv * (dk + dv) * e + B * (hq + hkv) * (dk + dv) * e,
                "flops": 2 * keys * hq * (dk + dv)}
    pairs = sum(min(p + 1, W) + min(ns, max(0, p + 1 - W)) for l in lengths for p in range(l))
    rows = B * L
    if kind == "win_forward":
        return {"bytes": e * tokens * ((hq + hkv) * dk + hkv * dv) + e * rows * hq * dv + 4 * rows * hq,
                "flops": 2 * pairs * hq * (dk + dv)}
    return {"bytes": e * (tokens * ((hq + hkv) * dk + (2 * hq + hkv) * dv) + rows * ((hq + hkv) * dk + hkv * dv))
            + 4 * rows * hq, "flops": 2 * pairs * hq * (3 * dk + 2 * dv)}


# ---- exact values -------------------------------------------------------------

def _exact_norm(case, s):
    x = s["x"].double()
    mean = x.sum(2) / case["D"]
    rstd = (((x - mean[:, :, None]) ** 2).sum(2) / case["D"] + EPS) ** -0.5
    if case["kind"] == "norm_forward":
        return {"y": torch.addcmul(s["bias"].double(), (x - mean[:, :, None]) * rstd[:, :, None], s["weight"].double()),
                "mean": mean, "rstd": rstd}
    mean, rstd = s["mean"].double()[:, :, None], s["rstd"].double()[:, :, None]
    xh, dy = (x - mean) * rstd, s["dy"].double()
    g = dy * s["weight"].double()
    share = (g.sum(2, keepdim=True) + xh * (g * xh).sum(2, keepdim=True)) / case["D"]
    return {"dx": rstd * (g - share), "dweight": (dy * xh).sum((0, 1)), "dbias": dy.sum((0, 1))}


def _exact_linear(case, s):
    """Position by position, in 64 bits."""
    B, H, scale = case["B"], case["heads"], case["d_k"] ** -0.5
    step = case["kind"] == "lin_step"
    q, k, v = ((s[n][:, None] if step else s[n]).double() for n in ("q", "k", "v"))
    L, decay = q.shape[1], s["log_decay"].double().exp()[:, None, None]
    S = torch.zeros((B, H, case["d_k"], case["d_v"]), dtype=torch.float64, device=q.device)
    if s["state"] is not None:
        S = s["state"].double()
    n = torch.tensor(_lengths(case), device=q.device)[:, None, None, None]
    grad = case["kind"] == "lin_backward"
    do = s["dout"].double() if grad else None
    out = torch.zeros(q.shape if grad else v.shape, dtype=torch.float64, device=q.device)
    for t in range(L):
        S = torch.where(t < n, decay * S + k[:, t, :, :, None] * v[:, t, :, None], S)
        out[:, t] = scale * ((S @ do[:, t, :, :, None])[..., 0] if grad else (q[:, t, :, None] @ S)[:, :, 0])
    here = torch.arange(L, device=q.device)[None, :, None, None] < n
    out = torch.where(here, out, 0.0)
    if not grad:
        return {"out": out[:, 0] if step else out, "state": S}
    dS = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in reversed(range(L)):
        new = dS + scale * q[:, t, :, :, None] * do[:, t, :, None]
        dk[:, t], dv[:, t] = (new @ v[:, t, :, :, None])[..., 0], (k[:, t, :, None] @ new)[:, :, 0]
        dS = torch.where(t < n, decay * new, dS)
    res = {"dq": out, "dk": torch.where(here, dk, 0.0), "dv": torch.where(here, dv, 0.0)}
    return res if s["state"] is None else {**res, "dstate": dS}


def _exact_window(case, s):
    """Head by head, in 64 bits, over all keys with the others left out."""
    L, G, ns, W = case["L"], case["heads_q"] // case["heads_kv"], case["n_sink"], case["window"]
    grad, dev = case["kind"] == "win_backward", s["q"].device
    out = torch.zeros((*s["q"].shape[:3], case["d_v"]), dtype=torch.float64, device=dev)
    lse = torch.full((case["B"], case["heads_q"], L), -math.inf, dtype=torch.float64, device=dev)
    dq, dk, dv = (torch.zeros(s[n].shape, dtype=torch.float64, device=dev) for n in ("q", "k", "v")) if grad \
        else (None,) * 3
    at = torch.arange(L, device=dev)
    back = at[:, None] - at  # how far a key lies behind the query
    hit = (back >= 0) & ((back < W) | (at < ns))
    for b, n in enumerate(_lengths(case)):
        for h in range(case["heads_q"]):
            q, k, v = s["q"][b, :n, h].double(), s["k"][b, :n, h // G].double(), s["v"][b, :n, h // G].double()
            score = (q @ k.T / math.sqrt(case["d_k"])).masked_fill(~hit[:n, :n], -math.inf)
            lse[b, h, :n] = torch.logsumexp(score, 1)
            p = (score - lse[b, h, :n, None]).exp()
            if not grad:
                out[b, :n, h] = p @ v
                continue
            do = s["dout"][b, :n, h].double()
            ds = p * (do @ v.T - (do * (p @ v)).sum(1, keepdim=True)) / math.sqrt(case["d_k"])
            dq[b, :n, h] = ds @ k
            dk[b, :n, h // G] += ds.T @ q
            dv[b, :n, h // G] += p.T @ do
    return {"dq": dq, "dk": dk, "dv": dv} if grad else {"out": out, "lse": lse}


def _exact_window_step(case, s):
    k, v, ns, G = s["k"], s["v"], case["n_sink"], case["heads_q"] // case["heads_kv"]
    room = _slots(case) - ns
    out = torch.zeros((case["B"], case["heads_q"], case["d_v"]), dtype=torch.float64, device=k.device)
    for b, n in enumerate(_lengths(case)):
        slots = [j if j < ns else ns + (j - ns) % room for j in range(n) if j < ns or j > n - 1 - case["window"]]
        k[b, slots[-1]], v[b, slots[-1]] = s["kt"][b], s["vt"][b]
        at = torch.tensor(slots, device=k.device)
        for h in range(case["heads_q"]):
            p = torch.softmax(k[b, at, h // G].double() @ s["q"][b, h].double() / math.sqrt(case["d_k"]), 0)
            out[b, h] = p @ v[b, at, h // G].double()
    return {"out": out, "k": k.double(), "v": v.double()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("norm"):
        return _exact_norm(case, s)
    if case["kind"].startswith("lin"):
        return _exact_linear(case, s)
    return _exact_window_step(case, s) if case["kind"] == "win_step" else _exact_window(case, s)
