"""How the attention weights' grids are split, told from the workspace's size (no GPU)."""
import pytest

from paged_kv_decode_21_gb300 import build as pkd_build


@pytest.fixture(scope="module")
def size():
    pkd_build.build()
    from paged_kv_decode_21_gb300 import ops
    return ops.paged_kv_attention_weights_workspace_size


def partitions(size, B, ql, Hq, H, most):
    """Partitions of a plan of more than 16 rows: two statistics of 4 bytes for every (b, g), partition and row."""
    rows = ql * Hq // H
    assert rows > 16 and B * H * rows * 4 % 256 == 0
    return size(B, ql, Hq, H, 128, 16, most) // (2 * 4 * B * H * rows)


@pytest.mark.parametrize("B,Hq,H,most", [(8, 32, 4, 16384), (4, 32, 8, 16384), (1, 32, 8, 16384), (32, 32, 8, 4096),
                                         (1, 16, 2, 8192), (64, 32, 8, 4096)])
def test_more_rows_do_not_leave_the_second_grid_fewer_ctas(size, B, Hq, H, most):
    """Its CTAs take all rows of a partition, so how many there are goes by sequences, heads and tokens alone."""
    few = partitions(size, B, 16, Hq, H, most)
    part = most // few
    for ql in (32, 64, 512, 2048):
        assert partitions(size, B, ql, Hq, H, most) in (few, min(few, most // 256)), ql
    # four for each SM at most, and more than half as many, where that leaves 256 to 4096 tokens a partition
    assert part == 4096 or B * H * few <= 4 * 152
    assert part <= 256 or 2 * B * H * few > 4 * 148
