"""Table builds at the limits of their sizes: the largest pool."""
import pytest

from step_harness import i32
from test_gpu_step import _cfg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("blocks", [2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 31])
def test_the_largest_pools(rbkv, blocks):
    """Blocks of one token, as many as a slot can number: the last ones are taken."""
    t = rbkv.StepTables(_cfg(rbkv, block=1, blocks=blocks), 2, 4, 8)
    t.free.zero_()
    t.free[-1] = 1 << ((blocks - 1) % 32) if (blocks - 1) % 32 < 31 else -2 ** 31
    t.free[-2] = 5
    first = (t.free.numel() - 2) * 32
    t.build(i32([0, 0]), i32([1, 2]))
    t.device_status()
    assert t.block_table[:, :2].tolist() == [[first, -1], [first + 2, blocks - 1]]
    assert t.slot.tolist() == [first, first + 2, blocks - 1, -1, -1, -1, -1, -1]
    assert not t.free.any()
    t.release(i32([0, 1]))
    t.device_status()
    assert t.free[-2].item() == 4 and t.free[-1].item() != 0
