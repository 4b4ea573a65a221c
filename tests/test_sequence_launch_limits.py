"""CPU: sizes within the documented limits that no launch can hold are refused before anything is enqueued.
The pointers are made up; where a GPU is there, nothing may get that far."""
import ctypes

import pytest

from scale_gla_layer_amd import binding as b
from scale_gla_layer_amd.config import BlockAttentionConfig, RecurrenceConfig

UNSUPPORTED, FAR = 2, 1 << 20
P = ctypes.c_void_p(FAR)


def _no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up pointers are for machines without a GPU")


def _rows():
    return b.CRows(FAR, 8192, 8192)


def _heads():
    return b.CHeads(FAR, 64, 64, 64)


def test_recurrence():
    _no_gpu()
    lib, big = b.load_library(), ctypes.c_size_t(-1)
    c = b.c_recurrence_config(RecurrenceConfig(8192, "norm"))
    assert lib.msgla_recurrence_forward(c, _rows(), _rows(), None, None, None, 1 << 17, 1, _rows(), None, P, big, None) == UNSUPPORTED
    assert lib.msgla_recurrence_backward(c, _rows(), _rows(), None, None, None, _rows(), None, 1 << 18, 1, _rows(), _rows(),
                                         None, None, P, big, None) == UNSUPPORTED
    c = b.c_recurrence_config(RecurrenceConfig(65536, "norm"))
    assert lib.msgla_recurrence_step(c, _rows(), _rows(), None, None, P, 1 << 17, _rows(), P, None) == UNSUPPORTED


def test_blocks():
    _no_gpu()
    lib, h, big = b.load_library(), _heads(), ctypes.c_size_t(-1)
    cfg = lambda heads: b.c_block_config(BlockAttentionConfig(heads, heads, 8, 8, 32, 1, 0, 1))  # noqa: E731
    assert lib.msgla_block_means(cfg(1), h, None, None, 1 << 10, 1 << 21, P, None) == UNSUPPORTED
    assert lib.msgla_block_select(cfg(16), h, P, None, None, 1, 1 << 24, 64, P, None) == UNSUPPORTED
    assert lib.msgla_block_attention(cfg(64), h, h, h, P, None, None, 1 << 20, 1, 64, h, P, P, big, None) == UNSUPPORTED
    assert lib.msgla_block_attention_backward(cfg(1), h, h, h, P, None, None, h, P, h, 256, 2, 1 << 21, h, h, h, P, big,
                                              None) == UNSUPPORTED
    assert lib.msgla_block_attention_step(cfg(8), h, h, h, P, 1 << 20, 64, h, h, P, h, P, big, None) == UNSUPPORTED
