"""CPU: layer norm, linear attention and window attention at sizes within the documented limits that no launch can
hold are refused before anything is enqueued.  The pointers are made up; where a GPU is there, nothing may get that far."""
import ctypes

from scale_gla_layer_amd import binding as b
from scale_gla_layer_amd.config import LayerNormConfig, LinearAttentionConfig, WindowAttentionConfig
from tests.test_sequence_launch_limits import UNSUPPORTED, P, _heads, _no_gpu

BIG = ctypes.c_size_t(-1)


def test_linear_attention():
    _no_gpu()
    lib, h = b.load_library(), _heads()
    for heads, dtype in ((64, "bf16"), (1024, "f32")):
        c = b.c_linear_config(LinearAttentionConfig(heads, 128, 256, dtype=dtype))
        B = 1 << 20
        assert lib.msgla_linear_attention_forward(c, h, h, h, P, None, None, B, 1, h, P, P, BIG, None) == UNSUPPORTED
        assert lib.msgla_linear_attention_backward(c, h, h, h, P, None, None, h, None, B, 1, h, h, h, None, P, BIG, None) == UNSUPPORTED
        assert lib.msgla_linear_attention_step(c, h, h, h, P, None, P, B, h, P, None) == UNSUPPORTED


def test_window_attention():
    _no_gpu()
    lib, h = b.load_library(), _heads()
    c = b.c_window_config(WindowAttentionConfig(1024, 1024, 64, 64, 100, 4))
    B = 1 << 20
    assert lib.msgla_window_attention(c, h, h, h, None, None, B, 1, 1, h, P, P, BIG, None) == UNSUPPORTED
    assert lib.msgla_window_attention_backward(c, h, h, h, None, None, h, P, h, B, 1, 1, h, h, h, P, BIG, None) == UNSUPPORTED
    assert lib.msgla_window_attention_append(c, h, h, None, None, B, 1 << 8, 1, h, h, None) == UNSUPPORTED
    assert lib.msgla_window_attention_step(c, h, h, h, P, B, 200, h, h, h, P, BIG, None) == UNSUPPORTED
    # few rows and a long cache: the rows' launches are small, the keys' are not
    c = b.c_window_config(WindowAttentionConfig(1024, 1024, 64, 64, 100, 4))
    assert lib.msgla_window_attention_backward(c, h, h, h, None, None, h, P, h, 64, 1, 1 << 24, h, h, h, P, BIG, None) == UNSUPPORTED


def test_sizes_at_their_ends():
    """Workspaces at the largest sizes are numbers that 64 bits hold, and what lies behind them is invalid."""
    bad, lib = 2 ** 64 - 1, b.load_library()
    c = b.c_layer_norm_config(LayerNormConfig(16384))
    assert 0 < lib.msgla_layer_norm_backward_workspace_bytes(c, 1 << 4, 1 << 24) < 1 << 40
    assert lib.msgla_layer_norm_backward_workspace_bytes(c, 1 << 5, 1 << 24) == bad
    c = b.c_linear_config(LinearAttentionConfig(1024, 256, 256))
    for f in (lib.msgla_linear_attention_workspace_bytes, lib.msgla_linear_attention_backward_workspace_bytes):
        assert f(c, 16, 1 << 24) < 1 << 50 and f(c, 1 << 20, 1 << 8) < 1 << 50 and f(c, 17, 1 << 24) == bad
    c = b.c_window_config(WindowAttentionConfig(1024, 1024, 128, 256, 1 << 24, 1024))
    for f in (lib.msgla_window_attention_workspace_bytes, lib.msgla_window_attention_backward_workspace_bytes):
        assert f(c, 16, 1 << 24, 1 << 24) < 1 << 60 and f(c, 17, 1 << 24, 1 << 24) == bad
    assert lib.msgla_window_attention_step_workspace_bytes(c, 1 << 20, 1 << 24) < 1 << 60
