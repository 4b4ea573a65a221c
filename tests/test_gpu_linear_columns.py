"""GPU: linear attention on either side of the size from which workgroups take 128 columns of the values, in many short
sequences and in a few long ones: ragged batches, states, widths that end inside the columns, against the 64-bit reference."""
import pytest

from tests.test_gpu_linear_attention import _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,L,H,dk,dv,lens,state", [
    (127, 65, 2, 128, 128, None, True),                                     # 254 walks: 64 columns
    (128, 65, 2, 128, 128, None, True),                                     # 256 walks
    (60, 130, 3, 72, 128, [(37 * b) % 131 for b in range(60)], True),
    (172, 40, 3, 96, 72, [(7 * b) % 42 for b in range(172)], False),
    (86, 64, 3, 128, 200, None, False),
    (1, 9000, 2, 128, 200, None, True),                                     # 564 chunks, in segments
    (2, 6000, 3, 80, 96, [6000, 4097], True),
    (1, 11000, 3, 40, 256, [10993], True)])                                 # keys of 64: 64 columns
def test_many_chunks(B, L, H, dk, dv, lens, state):
    _case(B, L, H, dk, dv, "bf16", lens, state)
