"""ctypes binding of libmsgla.so (include/msgla.h) — argument marshalling only.

Every function has the name of the C entry point it calls.  Device buffers
are torch tensors on a ROCm device (torch supplies the memory and the stream;
all computation happens in the library's HIP kernels).  A non-OK status
raises MsglaError.  Loading fails loudly when the library has not been built;
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

from .config import (BF16, F32, BlockAttentionConfig, LayerNormConfig, LinearAttentionConfig, MsglaConfig, RECURRENCE_INPUTS,
                     RecurrenceConfig, WindowAttentionConfig)

MAX_BRANCHES = 8
N_STAGES = 6
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmsgla.so")

STATUS = {0: "MSGLA_OK", 1: "MSGLA_ERR_INVALID_ARG", 2: "MSGLA_ERR_UNSUPPORTED",
          3: "MSGLA_ERR_WORKSPACE", 4: "MSGLA_ERR_HIP"}

# exported symbols declared by include/msgla.h
SYMBOLS = (
    "msgla_status_str", "msgla_validate_config", "msgla_packed_weights_bytes",
    "msgla_pack_weights", "msgla_workspace_bytes", "msgla_state_bytes", "msgla_state_init",
    "msgla_forward", "msgla_forward_timed", "msgla_decode_workspace_bytes", "msgla_decode_step",
    "msgla_fusion_weights", "msgla_state_query", "msgla_forward_noalloc",
    "msgla_backward_workspace_bytes", "msgla_backward", "msgla_forward_train", "msgla_backward_saved",
    "msgla_recurrence_workspace_bytes", "msgla_recurrence_backward_workspace_bytes",
    "msgla_recurrence_forward", "msgla_recurrence_backward", "msgla_recurrence_step",
    "msgla_block_means", "msgla_block_select", "msgla_block_attention_workspace_bytes",
    "msgla_block_attention_backward_workspace_bytes", "msgla_block_attention_step_workspace_bytes",
    "msgla_block_attention", "msgla_block_attention_backward", "msgla_block_attention_step",
    "msgla_layer_norm_backward_workspace_bytes", "msgla_layer_norm_forward", "msgla_layer_norm_backward",
    "msgla_linear_attention_workspace_bytes", "msgla_linear_attention_backward_workspace_bytes",
    "msgla_linear_attention_forward", "msgla_linear_attention_backward", "msgla_linear_attention_step",
    "msgla_window_attention_workspace_bytes", "msgla_window_attention_backward_workspace_bytes",
    "msgla_window_attention_step_workspace_bytes", "msgla_window_attention", "msgla_window_attention_backward",
    "msgla_window_attention_append", "msgla_window_attention_step",
)
NOALLOC_WORKSPACE_BYTES = 192 << 20  # MSGLA_NOALLOC_WORKSPACE_BYTES


class MsglaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")
        self.status = status


class CConfig(ctypes.Structure):
    _fields_ = [
        ("n_branches", ctypes.c_int32),
        ("scale", ctypes.c_int32 * MAX_BRANCHES),
        ("heads", ctypes.c_int32 * MAX_BRANCHES),
        ("d_model", ctypes.c_int32),
        ("d_k", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("gate_rank", ctypes.c_int32),
        ("chunk", ctypes.c_int32),
        ("gate_normalizer", ctypes.c_float),
        ("q_scale", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("norm", ctypes.c_int32),
    ]


class CBranchWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W_q", "W_k", "W_v", "W_g1", "W_g2", "b_g", "W_o",
                                               "norm_g")]


class CWeights(ctypes.Structure):
    _fields_ = [("br", CBranchWeights * MAX_BRANCHES), ("W_f", ctypes.c_void_p),
                ("b_f", ctypes.c_void_p)]


class CBranchGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W_q", "W_k", "W_v", "W_g1", "W_g2", "b_g", "W_o",
                                               "norm_g")]


class CGrads(ctypes.Structure):
    _fields_ = [("br", CBranchGrads * MAX_BRANCHES), ("W_f", ctypes.c_void_p),
                ("b_f", ctypes.c_void_p)]


class CStateInfo(ctypes.Structure):
    _fields_ = [("status", ctypes.c_int32), ("B", ctypes.c_int32), ("m", ctypes.c_int32),
                ("position", ctypes.c_int64)]


class CRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64)]


class CRecurrenceConfig(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("input", ctypes.c_int32), ("gate_normalizer", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class CHeads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


class CBlockConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads_q", "heads_kv", "d_k", "d_v", "block", "n_select", "n_first",
                                              "n_recent")] + [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class CLayerNormConfig(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


class CLinearConfig(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class CWindowConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads_q", "heads_kv", "d_k", "d_v", "window", "n_sink")] + \
        [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class CStageEvents(ctypes.Structure):
    _fields_ = [("start", ctypes.c_void_p * N_STAGES), ("stop", ctypes.c_void_p * N_STAGES)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmsgla.so; raises if it is missing (build it with scale_gla_layer_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run `python -m scale_gla_layer_amd.build` first "
                           "(the MS-GLA layer has no non-HIP implementation)")
    lib = ctypes.CDLL(path)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    cfgp = ctypes.POINTER(CConfig)
    sig = {
        "msgla_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "msgla_validate_config": (ctypes.c_int, [cfgp]),
        "msgla_packed_weights_bytes": (sz, [cfgp]),
        "msgla_pack_weights": (ctypes.c_int, [cfgp, ctypes.POINTER(CWeights), vp, sz, vp]),
        "msgla_workspace_bytes": (sz, [cfgp, i64, i64]),
        "msgla_state_bytes": (sz, [cfgp, i64]),
        "msgla_state_init": (ctypes.c_int, [cfgp, i64, vp, sz, vp]),
        "msgla_forward": (ctypes.c_int, [cfgp, vp, vp, vp, i64, i64, vp, vp, vp, vp, sz, vp]),
        "msgla_forward_timed": (ctypes.c_int, [cfgp, vp, vp, vp, i64, i64, vp, vp, vp, vp, sz, vp,
                                               ctypes.POINTER(CStageEvents)]),
        "msgla_decode_workspace_bytes": (sz, [cfgp, i64]),
        "msgla_decode_step": (ctypes.c_int, [cfgp, vp, vp, i64, vp, vp, vp, sz, vp]),
        "msgla_fusion_weights": (ctypes.c_int, [cfgp, vp, vp, i64, i64, vp, vp]),
        "msgla_state_query": (ctypes.c_int, [vp, ctypes.POINTER(CStateInfo), vp]),
        "msgla_forward_noalloc": (ctypes.c_int, [cfgp, vp, vp, vp, i64, i64, vp, vp, vp, vp]),
        "msgla_backward_workspace_bytes": (sz, [cfgp, i64, i64]),
        "msgla_backward": (ctypes.c_int, [cfgp, vp, vp, vp, vp, i64, i64, vp, ctypes.POINTER(CGrads),
                                          vp, sz, vp]),
        "msgla_backward_saved": (ctypes.c_int, [cfgp, vp, vp, vp, vp, i64, i64, vp, ctypes.POINTER(CGrads),
                                                vp, sz, vp]),
        "msgla_forward_train": (ctypes.c_int, [cfgp, vp, vp, vp, i64, i64, vp, vp, sz, vp]),
    }
    rows, rec = ctypes.POINTER(CRows), ctypes.POINTER(CRecurrenceConfig)
    sig.update({
        "msgla_recurrence_workspace_bytes": (sz, [rec, i64, i64]),
        "msgla_recurrence_backward_workspace_bytes": (sz, [rec, i64, i64]),
        "msgla_recurrence_forward": (ctypes.c_int, [rec, rows, rows, vp, vp, vp, i64, i64, rows, vp, vp, sz, vp]),
        "msgla_recurrence_backward": (ctypes.c_int, [rec, rows, rows, vp, vp, vp, rows, vp, i64, i64, rows, rows,
                                                     vp, vp, vp, sz, vp]),
        "msgla_recurrence_step": (ctypes.c_int, [rec, rows, rows, vp, vp, vp, i64, rows, vp, vp]),
    })
    heads, blk = ctypes.POINTER(CHeads), ctypes.POINTER(CBlockConfig)
    sig.update({
        "msgla_block_means": (ctypes.c_int, [blk, heads, vp, vp, i64, i64, vp, vp]),
        "msgla_block_select": (ctypes.c_int, [blk, heads, vp, vp, vp, i64, i64, i64, vp, vp]),
        "msgla_block_attention_workspace_bytes": (sz, [blk, i64, i64, i64]),
        "msgla_block_attention_backward_workspace_bytes": (sz, [blk, i64, i64, i64]),
        "msgla_block_attention_step_workspace_bytes": (sz, [blk, i64, i64]),
        "msgla_block_attention": (ctypes.c_int, [blk, heads, heads, heads, vp, vp, vp, i64, i64, i64, heads, vp, vp,
                                                 sz, vp]),
        "msgla_block_attention_backward": (ctypes.c_int, [blk, heads, heads, heads, vp, vp, vp, heads, vp, heads, i64,
                                                          i64, i64, heads, heads, heads, vp, sz, vp]),
        "msgla_block_attention_step": (ctypes.c_int, [blk, heads, heads, heads, vp, i64, i64, heads, heads, vp, heads,
                                                      vp, sz, vp]),
    })
    norm, lin = ctypes.POINTER(CLayerNormConfig), ctypes.POINTER(CLinearConfig)
    sig.update({
        "msgla_layer_norm_backward_workspace_bytes": (sz, [norm, i64, i64]),
        "msgla_layer_norm_forward": (ctypes.c_int, [norm, rows, vp, vp, i64, i64, rows, vp, vp, vp]),
        "msgla_layer_norm_backward": (ctypes.c_int, [norm, rows, rows, vp, vp, vp, i64, i64, rows, vp, vp, vp, sz, vp]),
        "msgla_linear_attention_workspace_bytes": (sz, [lin, i64, i64]),
        "msgla_linear_attention_backward_workspace_bytes": (sz, [lin, i64, i64]),
        "msgla_linear_attention_forward": (ctypes.c_int, [lin, heads, heads, heads, vp, vp, vp, i64, i64, heads, vp, vp,
                                                          sz, vp]),
        "msgla_linear_attention_backward": (ctypes.c_int, [lin, heads, heads, heads, vp, vp, vp, heads, vp, i64, i64,
                                                           heads, heads, heads, vp, vp, sz, vp]),
        "msgla_linear_attention_step": (ctypes.c_int, [lin, heads, heads, heads, vp, vp, vp, i64, heads, vp, vp]),
    })
    win = ctypes.POINTER(CWindowConfig)
    sig.update({
        "msgla_window_attention_workspace_bytes": (sz, [win, i64, i64, i64]),
        "msgla_window_attention_backward_workspace_bytes": (sz, [win, i64, i64, i64]),
        "msgla_window_attention_step_workspace_bytes": (sz, [win, i64, i64]),
        "msgla_window_attention": (ctypes.c_int, [win, heads, heads, heads, vp, vp, i64, i64, i64, heads, vp, vp, sz, vp]),
        "msgla_window_attention_backward": (ctypes.c_int, [win, heads, heads, heads, vp, vp, heads, vp, heads, i64, i64,
                                                           i64, heads, heads, heads, vp, sz, vp]),
        "msgla_window_attention_append": (ctypes.c_int, [win, heads, heads, vp, vp, i64, i64, i64, heads, heads, vp]),
        "msgla_window_attention_step": (ctypes.c_int, [win, heads, heads, heads, vp, i64, i64, heads, heads, heads, vp,
                                                       sz, vp]),
    })
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


_CFG_CACHE: dict = {}


def c_config(cfg: MsglaConfig) -> CConfig:
    """The C struct of a configuration (built once per distinct configuration)."""
    c = _CFG_CACHE.get(cfg)
    if c is None:
        c = _CFG_CACHE[cfg] = _build_config(cfg)
    return c


def _build_config(cfg: MsglaConfig) -> CConfig:
    c = CConfig()
    c.n_branches = len(cfg.scales)
    for i, (s, h) in enumerate(zip(cfg.scales, cfg.heads)):
        if i >= MAX_BRANCHES:
            break
        c.scale[i] = s
        c.heads[i] = h
    c.d_model, c.d_k, c.d_v = cfg.d_model, cfg.d_k, cfg.d_v
    c.gate_rank, c.chunk = cfg.gate_rank, cfg.chunk
    c.gate_normalizer, c.q_scale = cfg.gate_normalizer, cfg.q_scale
    c.dtype = 1 if cfg.dtype == BF16 else 0
    c.norm = 1 if cfg.norm else 0
    return c


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(fn: str, st: int):
    if st != 0:
        raise MsglaError(fn, st)


def msgla_validate_config(cfg: MsglaConfig) -> int:
    return load_library().msgla_validate_config(ctypes.byref(c_config(cfg)))


def msgla_packed_weights_bytes(cfg: MsglaConfig) -> int:
    return load_library().msgla_packed_weights_bytes(ctypes.byref(c_config(cfg)))


def msgla_workspace_bytes(cfg: MsglaConfig, B: int, L: int) -> int:
    return load_library().msgla_workspace_bytes(ctypes.byref(c_config(cfg)), B, L)


def msgla_state_bytes(cfg: MsglaConfig, B: int) -> int:
    return load_library().msgla_state_bytes(ctypes.byref(c_config(cfg)), B)


def msgla_decode_workspace_bytes(cfg: MsglaConfig, B: int) -> int:
    return load_library().msgla_decode_workspace_bytes(ctypes.byref(c_config(cfg)), B)


def msgla_pack_weights(cfg: MsglaConfig, branches: Sequence[dict], W_f, b_f, packed, stream=None):
    """branches: per branch a dict of device tensors W_q, W_k, W_v, W_g1, W_g2, b_g, W_o
    and, for configurations with the normalisation, norm_g."""
    w = CWeights()
    for i, br in enumerate(branches):
        for name in ("W_q", "W_k", "W_v", "W_g1", "W_g2", "b_g", "W_o", "norm_g"):
            setattr(w.br[i], name, _ptr(br.get(name)))
    w.W_f, w.b_f = _ptr(W_f), _ptr(b_f)
    st = load_library().msgla_pack_weights(ctypes.byref(c_config(cfg)), ctypes.byref(w),
                                           _ptr(packed), packed.numel() * packed.element_size(),
                                           _stream(stream))
    _check("msgla_pack_weights", st)


def msgla_state_init(cfg: MsglaConfig, B: int, state, stream=None):
    st = load_library().msgla_state_init(ctypes.byref(c_config(cfg)), B, _ptr(state),
                                         state.numel() * state.element_size(), _stream(stream))
    _check("msgla_state_init", st)


def msgla_forward(cfg: MsglaConfig, packed, x, B: int, L: int, out, workspace,
                  state_out=None, mask=None, state_in=None, stream=None, events=None):
    """events: optional (start[N_STAGES], stop[N_STAGES]) lists of torch.cuda.Event (or None entries)."""
    lib = load_library()
    args = (ctypes.byref(c_config(cfg)), _ptr(packed), _ptr(x), _ptr(mask), B, L, _ptr(out),
            _ptr(state_in), _ptr(state_out), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if events is None:
        st = lib.msgla_forward(*args)
        _check("msgla_forward", st)
        return
    ev = CStageEvents()
    for i in range(N_STAGES):
        for slot, lst in ((ev.start, events[0]), (ev.stop, events[1])):
            e = lst[i]
            slot[i] = None if e is None else e.cuda_event
    st = lib.msgla_forward_timed(*args, ctypes.byref(ev))
    _check("msgla_forward_timed", st)


def msgla_decode_step(cfg: MsglaConfig, packed, x_t, B: int, state, out_t, workspace, stream=None):
    st = load_library().msgla_decode_step(ctypes.byref(c_config(cfg)), _ptr(packed), _ptr(x_t), B,
                                          _ptr(state), _ptr(out_t), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _stream(stream))
    _check("msgla_decode_step", st)


def msgla_fusion_weights(cfg: MsglaConfig, packed, x, B: int, L: int, w_out, stream=None):
    st = load_library().msgla_fusion_weights(ctypes.byref(c_config(cfg)), _ptr(packed), _ptr(x), B, L,
                                             _ptr(w_out), _stream(stream))
    _check("msgla_fusion_weights", st)


def msgla_backward_workspace_bytes(cfg: MsglaConfig, B: int, L: int) -> int:
    return load_library().msgla_backward_workspace_bytes(ctypes.byref(c_config(cfg)), B, L)


def msgla_backward(cfg: MsglaConfig, packed, x, dout, B: int, L: int, dx, branch_grads: Sequence[dict],
                   W_f, b_f, workspace, mask=None, stream=None, saved=False):
    """branch_grads: per branch a dict of fp32 device tensors W_q, W_k, W_v, W_g1, W_g2, b_g, W_o
    and, for configurations with the normalisation, norm_g (written, in the layout of the
    weights); W_f, b_f: fp32 device tensors (None when m == 1);
    mask: the forward's [B, L] uint8 token mask, or None;
    saved: msgla_backward_saved (the workspace holds msgla_forward_train's intermediates)."""
    g = CGrads()
    for i, br in enumerate(branch_grads):
        for name in ("W_q", "W_k", "W_v", "W_g1", "W_g2", "b_g", "W_o", "norm_g"):
            setattr(g.br[i], name, _ptr(br.get(name)))
    g.W_f, g.b_f = _ptr(W_f), _ptr(b_f)
    name = "msgla_backward_saved" if saved else "msgla_backward"
    st = getattr(load_library(), name)(ctypes.byref(c_config(cfg)), _ptr(packed), _ptr(x), _ptr(dout),
                                       _ptr(mask), B, L, _ptr(dx), ctypes.byref(g), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check(name, st)


def msgla_forward_train(cfg: MsglaConfig, packed, x, B: int, L: int, out, workspace, mask=None, stream=None):
    """The training forward: out as msgla_forward, the backward's intermediates kept in
    workspace (at least msgla_backward_workspace_bytes)."""
    st = load_library().msgla_forward_train(ctypes.byref(c_config(cfg)), _ptr(packed), _ptr(x), _ptr(mask), B, L,
                                            _ptr(out), _ptr(workspace),
                                            workspace.numel() * workspace.element_size(), _stream(stream))
    _check("msgla_forward_train", st)


def msgla_state_query(state, stream=None) -> dict:
    """The state's header: {"status", "B", "m", "position"} (waits for the stream)."""
    info = CStateInfo()
    st = load_library().msgla_state_query(_ptr(state), ctypes.byref(info), _stream(stream))
    _check("msgla_state_query", st)
    return {"status": int(info.status), "B": int(info.B), "m": int(info.m),
            "position": int(info.position)}


def msgla_forward_noalloc(cfg: MsglaConfig, packed, x, B: int, L: int, out, state_out=None,
                          state_in=None, mask=None, stream=None):
    """The forward with the library's own per-device workspace (no allocation)."""
    st = load_library().msgla_forward_noalloc(ctypes.byref(c_config(cfg)), _ptr(packed), _ptr(x),
                                              _ptr(mask), B, L, _ptr(out), _ptr(state_in),
                                              _ptr(state_out), _stream(stream))
    _check("msgla_forward_noalloc", st)


# ---- sequence operators beside the layer ----------------------------------------
# Tensors are checked here against what the C entry points assume of the
# pointers they get; a ValueError names the argument.

_TORCH = None


def _t():
    """torch, imported at the first call."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _storage(cfg):
    return _t().bfloat16 if cfg.dtype == BF16 else _t().float32


def _raw_stream(stream) -> int:
    """The current stream of the current device, unless one is given."""
    if stream is not None:
        return _stream(stream)
    raw = getattr(_t()._C, "_cuda_getCurrentRawStream", None)  # without making a Stream object
    return _stream(None) if raw is None else raw(_t().cuda.current_device())


def _tensor(name: str, t, shape, dtype, device) -> tuple:
    """The strides of t, which has to have this shape (a tuple) and type on `device` (a ROCm device's)
    and dense rows in its last dimension."""
    strides = t.stride()
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and \
            (strides[-1] == 1 or shape[-1] == 1):
        return strides
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on {device}, a ROCm device: it is on {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}: it is {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}: it has {tuple(t.shape)}")
    raise ValueError(f"the last dimension of {name} must be dense")


def _dense(name: str, t, shape, dtype, device):
    """The address of a contiguous t, or None for None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _tensor(name, t, shape, dtype, device)
    raise ValueError(f"{name} must be contiguous")


def _f32(name: str, t, shape, device):
    return _dense(name, t, shape, _t().float32, device)


def _apart(name: str, t):
    """An output whose rows do not overlap (no broadcast dimension of more than one entry)."""
    if t.is_contiguous():
        return
    size = 1
    for n, s in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1), key=lambda p: p[1]):
        if s < size:
            raise ValueError(f"the rows of {name} overlap")
        size = s * (n - 1) + size


def _rows(name: str, t, shape, dtype, device) -> CRows:
    """[B, L, width], or [B, width] as rows of one position."""
    st = _tensor(name, t, shape, dtype, device)
    return CRows(t.data_ptr(), st[0], st[1] if len(st) == 3 else 0)


def _rows_out(name: str, t, shape, dtype, device) -> CRows:
    rows = _rows(name, t, shape, dtype, device)
    _apart(name, t)
    return rows


_REC_CACHE: dict = {}


def c_recurrence_config(cfg: RecurrenceConfig) -> CRecurrenceConfig:
    c = _REC_CACHE.get(cfg)
    if c is None:
        c = _REC_CACHE[cfg] = CRecurrenceConfig(cfg.width, RECURRENCE_INPUTS.index(cfg.input), cfg.gate_normalizer,
                                                1 if cfg.dtype == BF16 else 0)
    return c


def msgla_recurrence_workspace_bytes(cfg: RecurrenceConfig, B: int, L: int) -> int:
    return load_library().msgla_recurrence_workspace_bytes(ctypes.byref(c_recurrence_config(cfg)), B, L)


def msgla_recurrence_backward_workspace_bytes(cfg: RecurrenceConfig, B: int, L: int) -> int:
    return load_library().msgla_recurrence_backward_workspace_bytes(ctypes.byref(c_recurrence_config(cfg)), B, L)


def _recurrence_inputs(cfg, x, z, bias, mask, h_in, dims):
    """(shape, type, device, the C arguments of x, z, bias, mask and h_in)"""
    if x.dim() != dims:
        raise ValueError(f"x must have {dims} dimensions: it has {x.dim()}")
    shape, dt, dev = (*x.shape[:-1], cfg.width), _storage(cfg), x.device
    return shape, dt, dev, (_rows("x", x, shape, dt, dev), _rows("z", z, shape, dt, dev),
                            _f32("bias", bias, (cfg.width,), dev),
                            _dense("mask", mask, shape[:-1], _t().uint8, dev),
                            _f32("h_in", h_in, (shape[0], cfg.width), dev))


def _room(t, device) -> tuple:
    """Address and bytes of a workspace, which may be None."""
    if t is None:
        return None, 0
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}: it is on {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def msgla_recurrence_forward(cfg: RecurrenceConfig, x, z, y, workspace, bias=None, mask=None, h_in=None, h_out=None,
                             stream=None):
    """x, z, y: [B, L, width] (any strides with a dense last dimension); bias [width], h_in and h_out
    [B, width] fp32; mask: [B, L] uint8."""
    shape, dt, dev, args = _recurrence_inputs(cfg, x, z, bias, mask, h_in, 3)
    st = load_library().msgla_recurrence_forward(
        c_recurrence_config(cfg), *args, shape[0], shape[1], _rows_out("y", y, shape, dt, dev),
        _f32("h_out", h_out, (shape[0], cfg.width), dev), *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_recurrence_forward", st)


def msgla_recurrence_backward(cfg: RecurrenceConfig, x, z, dy, dx, dz, workspace, bias=None, mask=None, h_in=None,
                              dh_out=None, dbias=None, dh_in=None, stream=None):
    """dy (or None for 0), dx, dz: as x; dh_out, dh_in: [B, width] fp32; dbias: [width] fp32."""
    shape, dt, dev, args = _recurrence_inputs(cfg, x, z, bias, mask, h_in, 3)
    state = (shape[0], cfg.width)
    st = load_library().msgla_recurrence_backward(
        c_recurrence_config(cfg), *args, None if dy is None else _rows("dy", dy, shape, dt, dev),
        _f32("dh_out", dh_out, state, dev), shape[0], shape[1], _rows_out("dx", dx, shape, dt, dev),
        _rows_out("dz", dz, shape, dt, dev), _f32("dbias", dbias, (cfg.width,), dev), _f32("dh_in", dh_in, state, dev),
        *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_recurrence_backward", st)


def msgla_recurrence_step(cfg: RecurrenceConfig, x_t, z_t, y_t, h_in, h_out, bias=None, mask=None, stream=None):
    """x_t, z_t, y_t: [B, width]; h_in, h_out: [B, width] fp32 (may be one tensor); mask: [B] uint8."""
    shape, dt, dev, args = _recurrence_inputs(cfg, x_t, z_t, bias, mask, h_in, 2)
    st = load_library().msgla_recurrence_step(
        c_recurrence_config(cfg), *args, shape[0], _rows_out("y_t", y_t, shape, dt, dev),
        _f32("h_out", h_out, shape, dev), _raw_stream(stream))
    _check("msgla_recurrence_step", st)


def _heads(name: str, t, shape, dtype, device) -> CHeads:
    """[B, L, heads, width], or [B, heads, width] as rows of one position."""
    st = _tensor(name, t, shape, dtype, device)
    ptr, unit = t.data_ptr(), 16 // t.element_size()
    if (ptr % 16) or ((st[0] | st[1] | st[-2]) % unit):
        st = [0 if n == 1 else s for n, s in zip(shape, st)]
        if ptr % 16 or (st[0] | st[1] | st[-2]) % unit:
            raise ValueError(f"rows of {name} must start at multiples of 16 bytes")
    return CHeads(ptr, st[0], st[1] if len(st) == 4 else 0, st[-2])


def _heads_out(name: str, t, shape, dtype, device) -> CHeads:
    heads = _heads(name, t, shape, dtype, device)
    _apart(name, t)
    return heads


def _i32(name: str, t, shape, device):
    return _dense(name, t, shape, _t().int32, device)


_BLOCK_CACHE: dict = {}


def c_block_config(cfg: BlockAttentionConfig) -> CBlockConfig:
    c = _BLOCK_CACHE.get(cfg)
    if c is None:
        c = _BLOCK_CACHE[cfg] = CBlockConfig(cfg.heads_q, cfg.heads_kv, cfg.d_k, cfg.d_v, cfg.block, cfg.n_select,
                                             cfg.n_first, cfg.n_recent, cfg.scale, 1 if cfg.dtype == BF16 else 0)
    return c


def block_count(cfg: BlockAttentionConfig, S: int) -> int:
    return (S + cfg.block - 1) // cfg.block


def msgla_block_attention_workspace_bytes(cfg: BlockAttentionConfig, B: int, L: int, S: int) -> int:
    return load_library().msgla_block_attention_workspace_bytes(ctypes.byref(c_block_config(cfg)), B, L, S)


def msgla_block_attention_backward_workspace_bytes(cfg: BlockAttentionConfig, B: int, L: int, S: int) -> int:
    return load_library().msgla_block_attention_backward_workspace_bytes(ctypes.byref(c_block_config(cfg)), B, L, S)


def msgla_block_attention_step_workspace_bytes(cfg: BlockAttentionConfig, B: int, S: int) -> int:
    return load_library().msgla_block_attention_step_workspace_bytes(ctypes.byref(c_block_config(cfg)), B, S)


def _dims(name: str, t, n: int):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions: it has {t.dim()}")
    return t


def msgla_block_means(cfg: BlockAttentionConfig, k, means, lens=None, start_from=None, stream=None):
    """k [B, S, heads_kv, d_k] -> means [B, heads_kv, blocks, d_k] fp32; lens, start_from: [B] int32."""
    B, S, dev = *_dims("k", k, 4).shape[:2], k.device
    st = load_library().msgla_block_means(
        c_block_config(cfg), _heads("k", k, (B, S, cfg.heads_kv, cfg.d_k), _storage(cfg), dev),
        _i32("lens", lens, (B,), dev), _i32("start_from", start_from, (B,), dev), B, S,
        _f32("means", means, (B, cfg.heads_kv, block_count(cfg, S), cfg.d_k), dev), _raw_stream(stream))
    _check("msgla_block_means", st)


def msgla_block_select(cfg: BlockAttentionConfig, q, means, S: int, sel, start=None, lens=None, stream=None):
    """q [B, L, heads_q, d_k] -> sel [B, heads_kv, L, n_select] int32."""
    B, L, dev = *_dims("q", q, 4).shape[:2], q.device
    st = load_library().msgla_block_select(
        c_block_config(cfg), _heads("q", q, (B, L, cfg.heads_q, cfg.d_k), _storage(cfg), dev),
        _f32("means", means, (B, cfg.heads_kv, block_count(cfg, S), cfg.d_k), dev), _i32("start", start, (B,), dev),
        _i32("lens", lens, (B,), dev), B, L, S, _i32("sel", sel, (B, cfg.heads_kv, L, cfg.n_select), dev),
        _raw_stream(stream))
    _check("msgla_block_select", st)


def _block_inputs(cfg, q, k, v, sel, start, lens):
    """(B, L, S, type, device, the C arguments of the six)"""
    B, L = _dims("q", q, 4).shape[:2]
    S, dt, dev = _dims("k", k, 4).shape[1], _storage(cfg), q.device
    if sel is None:
        raise ValueError("sel is missing")
    return B, L, S, dt, dev, (
        _heads("q", q, (B, L, cfg.heads_q, cfg.d_k), dt, dev), _heads("k", k, (B, S, cfg.heads_kv, cfg.d_k), dt, dev),
        _heads("v", v, (B, S, cfg.heads_kv, cfg.d_v), dt, dev), _i32("sel", sel, (B, cfg.heads_kv, L, cfg.n_select), dev),
        _i32("start", start, (B,), dev), _i32("lens", lens, (B,), dev))


def msgla_block_attention(cfg: BlockAttentionConfig, q, k, v, sel, out, lse, workspace, start=None, lens=None,
                          stream=None):
    """q [B, L, heads_q, d_k], k [B, S, heads_kv, d_k], v [B, S, heads_kv, d_v] -> out [B, L, heads_q, d_v] and
    lse [B, heads_q, L] fp32 (or None)."""
    B, L, S, dt, dev, args = _block_inputs(cfg, q, k, v, sel, start, lens)
    st = load_library().msgla_block_attention(
        c_block_config(cfg), *args, B, L, S, _heads_out("out", out, (B, L, cfg.heads_q, cfg.d_v), dt, dev),
        _f32("lse", lse, (B, cfg.heads_q, L), dev), *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_block_attention", st)


def msgla_block_attention_backward(cfg: BlockAttentionConfig, q, k, v, sel, out, lse, dout, dq, dk, dv, workspace,
                                   start=None, lens=None, stream=None):
    B, L, S, dt, dev, args = _block_inputs(cfg, q, k, v, sel, start, lens)
    shape = (B, L, cfg.heads_q, cfg.d_v)
    st = load_library().msgla_block_attention_backward(
        c_block_config(cfg), *args, _heads("out", out, shape, dt, dev), _f32("lse", lse, (B, cfg.heads_q, L), dev),
        _heads("dout", dout, shape, dt, dev), B, L, S, _heads_out("dq", dq, tuple(q.shape), dt, dev),
        _heads_out("dk", dk, tuple(k.shape), dt, dev), _heads_out("dv", dv, tuple(v.shape), dt, dev),
        *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_block_attention_backward", st)


def msgla_block_attention_step(cfg: BlockAttentionConfig, q_t, k_t, v_t, k, v, means, pos, out_t, workspace,
                               stream=None):
    """q_t [B, heads_q, d_k], k_t [B, heads_kv, d_k], v_t [B, heads_kv, d_v], caches k [B, S, heads_kv, d_k] and
    v [B, S, heads_kv, d_v], means [B, heads_kv, blocks, d_k] fp32, pos [B] int32 -> out_t [B, heads_q, d_v]."""
    B, S, dt, dev = q_t.shape[0], _dims("k", k, 4).shape[1], _storage(cfg), q_t.device
    hq, hkv, dk, dv = cfg.heads_q, cfg.heads_kv, cfg.d_k, cfg.d_v
    st = load_library().msgla_block_attention_step(
        c_block_config(cfg), _heads("q_t", q_t, (B, hq, dk), dt, dev), _heads("k_t", k_t, (B, hkv, dk), dt, dev),
        _heads("v_t", v_t, (B, hkv, dv), dt, dev), _i32("pos", pos, (B,), dev), B, S,
        _heads_out("k", k, (B, S, hkv, dk), dt, dev), _heads_out("v", v, (B, S, hkv, dv), dt, dev),
        _f32("means", means, (B, hkv, block_count(cfg, S), dk), dev), _heads_out("out_t", out_t, (B, hq, dv), dt, dev),
        *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_block_attention_step", st)


_NORM_CACHE: dict = {}


def c_layer_norm_config(cfg: LayerNormConfig) -> CLayerNormConfig:
    c = _NORM_CACHE.get(cfg)
    if c is None:
        c = _NORM_CACHE[cfg] = CLayerNormConfig(cfg.width, cfg.eps, 1 if cfg.dtype == BF16 else 0)
    return c


def msgla_layer_norm_backward_workspace_bytes(cfg: LayerNormConfig, B: int, L: int) -> int:
    return load_library().msgla_layer_norm_backward_workspace_bytes(ctypes.byref(c_layer_norm_config(cfg)), B, L)


def msgla_layer_norm_forward(cfg: LayerNormConfig, x, y, weight=None, bias=None, mean=None, rstd=None, stream=None):
    """x, y: [B, L, width] (any strides with a dense last dimension); weight, bias [width] and mean, rstd [B, L] fp32."""
    B, L, dt, dev = *_dims("x", x, 3).shape[:2], _storage(cfg), x.device
    shape = (B, L, cfg.width)
    st = load_library().msgla_layer_norm_forward(
        c_layer_norm_config(cfg), _rows("x", x, shape, dt, dev), _f32("weight", weight, (cfg.width,), dev),
        _f32("bias", bias, (cfg.width,), dev), B, L, _rows_out("y", y, shape, dt, dev), _f32("mean", mean, (B, L), dev),
        _f32("rstd", rstd, (B, L), dev), _raw_stream(stream))
    _check("msgla_layer_norm_forward", st)


def msgla_layer_norm_backward(cfg: LayerNormConfig, x, dy, mean, rstd, dx, workspace, weight=None, dweight=None,
                              dbias=None, stream=None):
    """x, dy, dx: [B, L, width]; mean, rstd [B, L] and weight, dweight, dbias [width] fp32."""
    B, L, dt, dev = *_dims("x", x, 3).shape[:2], _storage(cfg), x.device
    shape = (B, L, cfg.width)
    st = load_library().msgla_layer_norm_backward(
        c_layer_norm_config(cfg), _rows("x", x, shape, dt, dev), _rows("dy", dy, shape, dt, dev),
        _f32("weight", weight, (cfg.width,), dev), _f32("mean", mean, (B, L), dev), _f32("rstd", rstd, (B, L), dev), B, L,
        _rows_out("dx", dx, shape, dt, dev), _f32("dweight", dweight, (cfg.width,), dev),
        _f32("dbias", dbias, (cfg.width,), dev), *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_layer_norm_backward", st)


_LINEAR_CACHE: dict = {}


def c_linear_config(cfg: LinearAttentionConfig) -> CLinearConfig:
    c = _LINEAR_CACHE.get(cfg)
    if c is None:
        c = _LINEAR_CACHE[cfg] = CLinearConfig(cfg.heads, cfg.d_k, cfg.d_v, cfg.scale, 1 if cfg.dtype == BF16 else 0)
    return c


def msgla_linear_attention_workspace_bytes(cfg: LinearAttentionConfig, B: int, L: int) -> int:
    return load_library().msgla_linear_attention_workspace_bytes(ctypes.byref(c_linear_config(cfg)), B, L)


def msgla_linear_attention_backward_workspace_bytes(cfg: LinearAttentionConfig, B: int, L: int) -> int:
    return load_library().msgla_linear_attention_backward_workspace_bytes(ctypes.byref(c_linear_config(cfg)), B, L)


def _state(name: str, t, cfg, B: int, device):
    p = _f32(name, t, (B, cfg.heads, cfg.d_k, cfg.d_v), device)
    if p is not None and p % 16:
        raise ValueError(f"{name} must start at a multiple of 16 bytes")
    return p


def _decay(t, cfg, device):
    if t is None:
        raise ValueError("log_decay is missing")
    return _f32("log_decay", t, (cfg.heads,), device)


def _linear_inputs(cfg, q, k, v, log_decay, lens, state_in):
    """(B, L, type, device, the C arguments of the six)"""
    B, L, dt, dev = *_dims("q", q, 4).shape[:2], _storage(cfg), q.device
    key, value = (B, L, cfg.heads, cfg.d_k), (B, L, cfg.heads, cfg.d_v)
    return B, L, dt, dev, (_heads("q", q, key, dt, dev), _heads("k", k, key, dt, dev), _heads("v", v, value, dt, dev),
                           _decay(log_decay, cfg, dev), _i32("lens", lens, (B,), dev),
                           _state("state_in", state_in, cfg, B, dev))


def msgla_linear_attention_forward(cfg: LinearAttentionConfig, q, k, v, log_decay, out, workspace, lens=None,
                                   state_in=None, state_out=None, stream=None):
    """q, k [B, L, heads, d_k], v [B, L, heads, d_v], log_decay [heads] fp32 -> out [B, L, heads, d_v]; lens [B] int32;
    state_in, state_out [B, heads, d_k, d_v] fp32 (may be one tensor)."""
    B, L, dt, dev, args = _linear_inputs(cfg, q, k, v, log_decay, lens, state_in)
    st = load_library().msgla_linear_attention_forward(
        c_linear_config(cfg), *args, B, L, _heads_out("out", out, (B, L, cfg.heads, cfg.d_v), dt, dev),
        _state("state_out", state_out, cfg, B, dev), *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_linear_attention_forward", st)


def msgla_linear_attention_backward(cfg: LinearAttentionConfig, q, k, v, log_decay, dout, dq, dk, dv, workspace,
                                    lens=None, state_in=None, dstate_out=None, dstate_in=None, stream=None):
    B, L, dt, dev, args = _linear_inputs(cfg, q, k, v, log_decay, lens, state_in)
    key, value = (B, L, cfg.heads, cfg.d_k), (B, L, cfg.heads, cfg.d_v)
    st = load_library().msgla_linear_attention_backward(
        c_linear_config(cfg), *args, _heads("dout", dout, value, dt, dev), _state("dstate_out", dstate_out, cfg, B, dev),
        B, L, _heads_out("dq", dq, key, dt, dev), _heads_out("dk", dk, key, dt, dev),
        _heads_out("dv", dv, value, dt, dev), _state("dstate_in", dstate_in, cfg, B, dev), *_room(workspace, dev),
        _raw_stream(stream))
    _check("msgla_linear_attention_backward", st)


def msgla_linear_attention_step(cfg: LinearAttentionConfig, q_t, k_t, v_t, log_decay, state_in, state_out, out_t,
                                mask=None, stream=None):
    """q_t, k_t [B, heads, d_k], v_t [B, heads, d_v] -> out_t [B, heads, d_v]; state_in, state_out [B, heads, d_k, d_v]
    fp32 (may be one tensor); mask: [B] uint8."""
    B, dt, dev = _dims("q_t", q_t, 3).shape[0], _storage(cfg), q_t.device
    key, value = (B, cfg.heads, cfg.d_k), (B, cfg.heads, cfg.d_v)
    st = load_library().msgla_linear_attention_step(
        c_linear_config(cfg), _heads("q_t", q_t, key, dt, dev), _heads("k_t", k_t, key, dt, dev),
        _heads("v_t", v_t, value, dt, dev), _decay(log_decay, cfg, dev), _dense("mask", mask, (B,), _t().uint8, dev),
        _state("state_in", state_in, cfg, B, dev), B, _heads_out("out_t", out_t, value, dt, dev),
        _state("state_out", state_out, cfg, B, dev), _raw_stream(stream))
    _check("msgla_linear_attention_step", st)


_WINDOW_CACHE: dict = {}


def c_window_config(cfg: WindowAttentionConfig) -> CWindowConfig:
    c = _WINDOW_CACHE.get(cfg)
    if c is None:
        c = _WINDOW_CACHE[cfg] = CWindowConfig(cfg.heads_q, cfg.heads_kv, cfg.d_k, cfg.d_v, cfg.window, cfg.n_sink,
                                               cfg.scale, 1 if cfg.dtype == BF16 else 0)
    return c


def msgla_window_attention_workspace_bytes(cfg: WindowAttentionConfig, B: int, L: int, S: int) -> int:
    return load_library().msgla_window_attention_workspace_bytes(ctypes.byref(c_window_config(cfg)), B, L, S)


def msgla_window_attention_backward_workspace_bytes(cfg: WindowAttentionConfig, B: int, L: int, S: int) -> int:
    return load_library().msgla_window_attention_backward_workspace_bytes(ctypes.byref(c_window_config(cfg)), B, L, S)


def msgla_window_attention_step_workspace_bytes(cfg: WindowAttentionConfig, B: int, S: int) -> int:
    return load_library().msgla_window_attention_step_workspace_bytes(ctypes.byref(c_window_config(cfg)), B, S)


def _window_inputs(cfg, q, k, v, start, lens):
    """(B, L, S, type, device, the C arguments of the five)"""
    B, L = _dims("q", q, 4).shape[:2]
    S, dt, dev = _dims("k", k, 4).shape[1], _storage(cfg), q.device
    return B, L, S, dt, dev, (
        _heads("q", q, (B, L, cfg.heads_q, cfg.d_k), dt, dev), _heads("k", k, (B, S, cfg.heads_kv, cfg.d_k), dt, dev),
        _heads("v", v, (B, S, cfg.heads_kv, cfg.d_v), dt, dev), _i32("start", start, (B,), dev),
        _i32("lens", lens, (B,), dev))


def msgla_window_attention(cfg: WindowAttentionConfig, q, k, v, out, lse, workspace, start=None, lens=None, stream=None):
    """q [B, L, heads_q, d_k], k [B, S, heads_kv, d_k], v [B, S, heads_kv, d_v] -> out [B, L, heads_q, d_v] and
    lse [B, heads_q, L] fp32 (or None); start, lens: [B] int32."""
    B, L, S, dt, dev, args = _window_inputs(cfg, q, k, v, start, lens)
    st = load_library().msgla_window_attention(
        c_window_config(cfg), *args, B, L, S, _heads_out("out", out, (B, L, cfg.heads_q, cfg.d_v), dt, dev),
        _f32("lse", lse, (B, cfg.heads_q, L), dev), *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_window_attention", st)


def msgla_window_attention_backward(cfg: WindowAttentionConfig, q, k, v, out, lse, dout, dq, dk, dv, workspace,
                                    start=None, lens=None, stream=None):
    B, L, S, dt, dev, args = _window_inputs(cfg, q, k, v, start, lens)
    shape = (B, L, cfg.heads_q, cfg.d_v)
    st = load_library().msgla_window_attention_backward(
        c_window_config(cfg), *args, _heads("out", out, shape, dt, dev), _f32("lse", lse, (B, cfg.heads_q, L), dev),
        _heads("dout", dout, shape, dt, dev), B, L, S, _heads_out("dq", dq, tuple(q.shape), dt, dev),
        _heads_out("dk", dk, tuple(k.shape), dt, dev), _heads_out("dv", dv, tuple(v.shape), dt, dev),
        *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_window_attention_backward", st)


def msgla_window_attention_append(cfg: WindowAttentionConfig, k_new, v_new, k, v, pos=None, lens=None, stream=None):
    """k_new [B, L, heads_kv, d_k], v_new [B, L, heads_kv, d_v] into the caches k [B, S, heads_kv, d_k] and
    v [B, S, heads_kv, d_v] at positions pos [B] int32 (None: 0) and on; lens [B] int32: new tokens of each sequence."""
    B, L = _dims("k_new", k_new, 4).shape[:2]
    S, dt, dev, H = _dims("k", k, 4).shape[1], _storage(cfg), k_new.device, cfg.heads_kv
    st = load_library().msgla_window_attention_append(
        c_window_config(cfg), _heads("k_new", k_new, (B, L, H, cfg.d_k), dt, dev),
        _heads("v_new", v_new, (B, L, H, cfg.d_v), dt, dev), _i32("pos", pos, (B,), dev), _i32("lens", lens, (B,), dev),
        B, L, S, _heads_out("k", k, (B, S, H, cfg.d_k), dt, dev), _heads_out("v", v, (B, S, H, cfg.d_v), dt, dev),
        _raw_stream(stream))
    _check("msgla_window_attention_append", st)


def msgla_window_attention_step(cfg: WindowAttentionConfig, q_t, k_t, v_t, k, v, pos, out_t, workspace, stream=None):
    """q_t [B, heads_q, d_k], k_t [B, heads_kv, d_k], v_t [B, heads_kv, d_v], caches k [B, S, heads_kv, d_k] and
    v [B, S, heads_kv, d_v], pos [B] int32 -> out_t [B, heads_q, d_v]."""
    B, S, dt, dev = _dims("q_t", q_t, 3).shape[0], _dims("k", k, 4).shape[1], _storage(cfg), q_t.device
    hq, hkv, dk, dv = cfg.heads_q, cfg.heads_kv, cfg.d_k, cfg.d_v
    st = load_library().msgla_window_attention_step(
        c_window_config(cfg), _heads("q_t", q_t, (B, hq, dk), dt, dev), _heads("k_t", k_t, (B, hkv, dk), dt, dev),
        _heads("v_t", v_t, (B, hkv, dv), dt, dev), _i32("pos", pos, (B,), dev), B, S,
        _heads_out("k", k, (B, S, hkv, dk), dt, dev), _heads_out("v", v, (B, S, hkv, dv), dt, dev),
        _heads_out("out_t", out_t, (B, hq, dv), dt, dev), *_room(workspace, dev), _raw_stream(stream))
    _check("msgla_window_attention_step", st)
