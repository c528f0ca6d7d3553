"""Rules of the adapter calls that the workspace sizes show; no device is touched."""
import pytest


@pytest.mark.parametrize("groups", [16, 64, 128, 512, 4096])
@pytest.mark.parametrize("r,N", [(16, 4096), (32, 2048), (32, 512)])
def test_a_long_group_is_cut_however_many_groups_there_are(e4b, groups, r, N):
    """Only the parts of groups of several tiles are kept; without gx and ga the workspace is those of
    gb.  A quarter of the 512 workgroups a pass is given, or 128 rows a tile, is room enough for a group
    with half of the rows to be shared out."""
    S = 16384
    parts = e4b.e4b_lora_backward_workspace_bytes(S, 64, N, r, groups, groups, gx=False, ga=False) // (4 * r * N)
    assert parts >= min(512 // (N // 256) // 4, S // 128 // 2)
