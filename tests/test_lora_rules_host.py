"""Rules of the adapter calls that the workspace sizes show; no device is touched."""
import ctypes

import pytest

from test_lora_host import ERR_OVERFLOW, _backward, _forward


@pytest.mark.parametrize("groups", [16, 64, 128, 512, 4096])
@pytest.mark.parametrize("r,N", [(16, 4096), (32, 2048), (32, 512)])
def test_a_long_group_is_cut_however_many_groups_there_are(e4b, groups, r, N):
    """Only the parts of groups of several tiles are kept; without gx and ga the workspace is those of
    gb.  A quarter of the 512 workgroups a pass is given, or 128 rows a tile, is room enough for a group
    with half of the rows to be shared out."""
    S = 16384
    parts = e4b.e4b_lora_backward_workspace_bytes(S, 64, N, r, groups, groups, gx=False, ga=False) // (4 * r * N)
    assert parts >= min(512 // (N // 256) // 4, S // 128 // 2)


def test_groups_are_limited(e4b):
    """Every workgroup reads the groups in turn: a call over millions of them would not end in any useful time."""
    for groups, status in ((65536, 0), (65537, ERR_OVERFLOW), (1 << 22, ERR_OVERFLOW), ((1 << 31) - 1, ERR_OVERFLOW)):
        n = ctypes.c_size_t(0)
        assert e4b._c_lora_ws(ctypes.byref(_forward(e4b, S=groups, groups=groups)), ctypes.byref(n)) == status
        assert e4b._c_lora_bwd_ws(ctypes.byref(_backward(e4b, S=groups, groups=groups)), ctypes.byref(n)) == status
    assert e4b._c_lora(ctypes.byref(_forward(e4b, groups=65537)), None) == ERR_OVERFLOW
    assert e4b._c_lora_bwd(ctypes.byref(_backward(e4b, groups=65537)), None) == ERR_OVERFLOW
