"""Layer configuration and the named synthetic workloads.

The layer is the MS-GLA token-mixing layer described in the reading notes
"MS-GLA：多时间尺度门控线性注意力研读笔记" (notes on arXiv:2609.35664,
"MS-GLA: Multi-Scale Gated Linear Attention ..."), Sec. 3 and Eqs. (8)-(11).

A configuration names a set of branches.  Branch i pools the sequence over
non-overlapping blocks of ``scales[i]`` tokens and owns ``heads[i]`` GLA heads
of width ``d_k`` x ``d_v`` (Sec. 3.2, Eq. (9): the head counts add up to the
layer's total H).  ``gate_rank`` is the rank r of the low-rank forget-gate
projection, ``gate_normalizer`` the divisor applied to logsigmoid, and
``chunk`` is only the GPU schedule's chunk length (Sec. 3.4 separates the
pooling block from the kernel chunk; results do not depend on it).
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Tuple

F32 = "f32"
BF16 = "bf16"


@dataclasses.dataclass(frozen=True)
class MsglaConfig:
    scales: Tuple[int, ...]
    heads: Tuple[int, ...]
    d_model: int
    d_k: int
    d_v: int
    gate_rank: int
    chunk: int = 64
    gate_normalizer: float = 16.0
    q_scale: float = 1.0
    dtype: str = BF16
    norm: bool = False  # per-head RMS normalisation of each branch's output before W_o

    def __post_init__(self):
        if len(self.scales) != len(self.heads) or not self.scales:
            raise ValueError("scales and heads must be non-empty and of equal length")
        if len(set(self.scales)) != len(self.scales):
            raise ValueError("scales must be distinct")
        if any(s <= 0 for s in self.scales) or any(h <= 0 for h in self.heads):
            raise ValueError("scales and heads must be positive")
        if self.dtype not in (F32, BF16):
            raise ValueError(f"dtype must be {F32!r} or {BF16!r}")

    @property
    def n_branches(self) -> int:
        return len(self.scales)

    @property
    def total_heads(self) -> int:
        return sum(self.heads)

    def state_elements(self) -> int:
        """Recurrent-state elements per sequence: sum_s h_s d_k d_v = H d_k d_v."""
        return sum(h * self.d_k * self.d_v for h in self.heads)


RECURRENCE_INPUTS = ("plain", "convex", "norm")


@dataclasses.dataclass(frozen=True)
class RecurrenceConfig:
    """Gated linear recurrence h_t = alpha_t h_{t-1} + beta_t x_t per channel, with
    log alpha_t = logsigmoid(z_t + bias) / gate_normalizer and beta 1 ("plain"),
    1 - alpha ("convex") or sqrt(1 - alpha^2) ("norm")."""
    width: int
    input: str = "plain"
    gate_normalizer: float = 16.0
    dtype: str = BF16

    def __post_init__(self):
        if not 1 <= self.width <= 65536:
            raise ValueError("width must be 1 .. 65536")
        if self.input not in RECURRENCE_INPUTS:
            raise ValueError(f"input must be one of {RECURRENCE_INPUTS}")
        if not 1e-6 <= self.gate_normalizer <= 1e6:
            raise ValueError("gate_normalizer must be 1e-6 .. 1e6")
        if self.dtype not in (F32, BF16):
            raise ValueError(f"dtype must be {F32!r} or {BF16!r}")


@dataclasses.dataclass(frozen=True)
class BlockAttentionConfig:
    """Attention over selected blocks of keys: each query attends the first ``n_first`` blocks of
    ``block`` positions, the ``n_recent`` ones that end with its own, and those whose mean key scores
    highest against the sum of its group's queries, ``n_select`` in all.  ``scale`` None: 1 / sqrt(d_k)."""
    heads_q: int
    heads_kv: int
    d_k: int
    d_v: int
    block: int = 64
    n_select: int = 16
    n_first: int = 1
    n_recent: int = 2
    scale: Optional[float] = None
    dtype: str = BF16

    def __post_init__(self):
        if self.heads_kv < 1 or not self.heads_kv <= self.heads_q <= 1024 or self.heads_q % self.heads_kv:
            raise ValueError("heads_q must be a multiple of heads_kv, at most 1024")
        if not 8 <= self.d_k <= 128 or self.d_k % 8 or not 8 <= self.d_v <= 256 or self.d_v % 8:
            raise ValueError("d_k must be a multiple of 8 up to 128, d_v one up to 256")
        if self.block not in (32, 64, 128):
            raise ValueError("block must be 32, 64 or 128")
        if not 1 <= self.n_select <= 64:
            raise ValueError("n_select must be 1 .. 64")
        if self.n_first < 0 or self.n_recent < 1 or self.n_first + self.n_recent > self.n_select:
            raise ValueError("n_first >= 0, n_recent >= 1 and n_first + n_recent <= n_select are required")
        if self.scale is None:
            object.__setattr__(self, "scale", self.d_k ** -0.5)
        if not 1e-30 <= self.scale <= 1e30:
            raise ValueError("scale must be positive, 1e-30 .. 1e30")
        if self.dtype not in (F32, BF16):
            raise ValueError(f"dtype must be {F32!r} or {BF16!r}")


@dataclasses.dataclass(frozen=True)
class LayerNormConfig:
    """Layer norm over the last dimension: (x - mean) / sqrt(variance + eps), times a weight, plus a bias."""
    width: int
    eps: float = 1e-5
    dtype: str = BF16

    def __post_init__(self):
        if not 1 <= self.width <= 16384:
            raise ValueError("width must be 1 .. 16384")
        if not 1e-20 <= self.eps <= 1:
            raise ValueError("eps must be 1e-20 .. 1")
        if self.dtype not in (F32, BF16):
            raise ValueError(f"dtype must be {F32!r} or {BF16!r}")


@dataclasses.dataclass(frozen=True)
class LinearAttentionConfig:
    """Linear attention with a decay for each head: S_t = gamma S_{t-1} + k_t^T v_t, out_t = scale q_t S_t.
    ``scale`` None: 1 / sqrt(d_k)."""
    heads: int
    d_k: int
    d_v: int
    scale: Optional[float] = None
    dtype: str = BF16

    def __post_init__(self):
        if not 1 <= self.heads <= 1024:
            raise ValueError("heads must be 1 .. 1024")
        if not 8 <= self.d_k <= 256 or self.d_k % 8 or not 8 <= self.d_v <= 256 or self.d_v % 8:
            raise ValueError("d_k and d_v must be multiples of 8 up to 256")
        if self.scale is None:
            object.__setattr__(self, "scale", self.d_k ** -0.5)
        if not 1e-30 <= self.scale <= 1e30:
            raise ValueError("scale must be positive, 1e-30 .. 1e30")
        if self.dtype not in (F32, BF16):
            raise ValueError(f"dtype must be {F32!r} or {BF16!r}")


@dataclasses.dataclass(frozen=True)
class WindowAttentionConfig:
    """Attention with a sliding window: a query at position p attends the keys j <= p with j > p - ``window`` or
    j < ``n_sink``, the first tokens that stay visible.  ``scale`` None: 1 / sqrt(d_k)."""
    heads_q: int
    heads_kv: int
    d_k: int
    d_v: int
    window: int
    n_sink: int = 0
    scale: Optional[float] = None
    dtype: str = BF16

    def __post_init__(self):
        if self.heads_kv < 1 or not self.heads_kv <= self.heads_q <= 1024 or self.heads_q % self.heads_kv:
            raise ValueError("heads_q must be a multiple of heads_kv, at most 1024")
        if not 8 <= self.d_k <= 128 or self.d_k % 8 or not 8 <= self.d_v <= 256 or self.d_v % 8:
            raise ValueError("d_k must be a multiple of 8 up to 128, d_v one up to 256")
        if not 1 <= self.window <= 1 << 24:
            raise ValueError("window must be 1 .. 2^24")
        if not 0 <= self.n_sink <= 1024:
            raise ValueError("n_sink must be 0 .. 1024")
        if self.scale is None:
            object.__setattr__(self, "scale", self.d_k ** -0.5)
        if not 1e-30 <= self.scale <= 1e30:
            raise ValueError("scale must be positive, 1e-30 .. 1e30")
        if self.dtype not in (F32, BF16):
            raise ValueError(f"dtype must be {F32!r} or {BF16!r}")


@dataclasses.dataclass(frozen=True)
class Workload:
    name: str
    cfg: MsglaConfig
    batch: int
    seq_len: int
    gate_bias: Optional[Tuple[float, float]] = None  # U(lo, hi) per channel, else 0
    description: str = ""


def _layer(scales, heads, dtype=BF16, d=1024, dk=128, dv=256, r=16, chunk=64):
    return MsglaConfig(tuple(scales), tuple(heads), d, dk, dv, r, chunk, 16.0, 1.0, dtype)


WORKLOADS = {
    "tiny_f32": Workload(
        "tiny_f32", MsglaConfig((1, 2, 4), (2, 1, 1), 64, 16, 32, 4, 16, 16.0, 1.0, F32),
        batch=1, seq_len=64,
        description="tiny fp32 MS-GLA {1,2,4}/[2,1,1], d=64, d_k=16, d_v=32, r=4, chunk 16"),
    "gla_baseline": Workload(
        "gla_baseline", _layer((1,), (4,)), batch=8, seq_len=2048,
        description="single-scale GLA layer, 4 heads at scale 1, B=8, L=2048, d=1024, bf16"),
    "main": Workload(
        "main", _layer((1, 2, 4), (2, 1, 1)), batch=8, seq_len=2048,
        description="MS-GLA {1,2,4}/[2,1,1], B=8, L=2048, d=1024, bf16"),
    "long": Workload(
        "long", _layer((1, 2, 4), (2, 1, 1)), batch=1, seq_len=16384, gate_bias=(1.0, 4.0),
        description="MS-GLA {1,2,4}/[2,1,1], B=1, L=16384, gate bias U(1,4), bf16"),
    "sweep_1248": Workload(
        "sweep_1248", _layer((1, 2, 4, 8), (1, 1, 1, 1)), batch=16, seq_len=4096,
        description="MS-GLA {1,2,4,8}/[1,1,1,1], B=16, L=4096, bf16"),
    "sweep_24": Workload(
        "sweep_24", _layer((2, 4), (2, 2)), batch=16, seq_len=4096,
        description="MS-GLA {2,4}/[2,2] (no fine branch), B=16, L=4096, bf16"),
}
