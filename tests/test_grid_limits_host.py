"""Sizes whose grids a launch cannot have are refused before anything is enqueued: HIP takes fewer
than 2^32 work items (workgroups times threads of one) a dimension.  No device is touched."""
import ctypes

import pytest

from test_lora_host import ERR_OVERFLOW, ERR_WORKSPACE, FAKE, _backward, _forward

BF16, F32 = 0, 1
ROOM = 1 << 50  # bytes of a workspace that is never looked into


def _permute(e4b, T, H, k, dtype=BF16, n=0):
    return e4b._c_permute(FAKE, dtype, T, H, k, FAKE, FAKE, FAKE, n, None)


def _combine(e4b, T, H, k, dtype=F32, n=0):
    return e4b._c_combine(FAKE, dtype, T, H, k, FAKE, FAKE, FAKE, BF16, FAKE, n, None)


def _combine_bwd(e4b, T, H, k, n=0):
    return e4b._c_combine_bwd(FAKE, BF16, FAKE, F32, T, H, k, FAKE, FAKE, FAKE, BF16, FAKE, FAKE, n, None)


# Each size at the limit, and one step below it (accepted up to the workspace, which is missing, or up
# to the device).  A gathered row of 512 bf16 and more is a wave's: 2^26 rows are 2^32 lanes.
def test_gathered_rows(e4b):
    n = ctypes.c_size_t(0)
    for T in (1 << 26, 1 << 27):
        assert _permute(e4b, T, 512, 1) == ERR_OVERFLOW and _permute(e4b, T, 4096, 1) == ERR_OVERFLOW
        assert e4b._c_permute_ws(BF16, T, 512, 1, ctypes.byref(n)) == ERR_OVERFLOW
    assert e4b._c_permute_ws(BF16, (1 << 26) - 4, 4096, 1, ctypes.byref(n)) == 0
    # 257 bf16 columns: a wave (33 pieces of 16 bytes); 256: 32 lanes
    assert e4b._c_permute_ws(BF16, 1 << 26, 257, 1, ctypes.byref(n)) == ERR_OVERFLOW
    assert e4b._c_permute_ws(BF16, 1 << 26, 256, 1, ctypes.byref(n)) == 0
    assert e4b._c_permute_ws(F32, 1 << 26, 129, 1, ctypes.byref(n)) == ERR_OVERFLOW
    assert e4b._c_permute_ws(F32, 1 << 26, 128, 1, ctypes.byref(n)) == 0


def test_rows_in_token_order(e4b):
    """k > 1: 16 bytes a lane of x, and behind them a lane for each row."""
    n = ctypes.c_size_t(0)
    assert e4b._c_permute_ws(BF16, 1 << 26, 512, 2, ctypes.byref(n)) == ERR_OVERFLOW
    assert e4b._c_permute_ws(BF16, 1 << 23, 4096, 8, ctypes.byref(n)) == ERR_OVERFLOW
    assert e4b._c_permute_ws(BF16, 1 << 22, 4096, 8, ctypes.byref(n)) == 0 and n.value >= 4 << 25


def test_combined_rows(e4b):
    # 4 float32 or 8 bf16 columns a lane
    assert _combine(e4b, 1 << 22, 4096, 2) == ERR_OVERFLOW and _combine(e4b, 1 << 21, 4096, 2) == ERR_WORKSPACE
    assert _combine(e4b, 1 << 23, 4096, 2, BF16) == ERR_OVERFLOW and _combine(e4b, 1 << 22, 4096, 2, BF16) == ERR_WORKSPACE
    # a wave for each row of the gradient
    assert _combine_bwd(e4b, 1 << 25, 512, 2) == ERR_OVERFLOW and _combine_bwd(e4b, (1 << 25) - 8, 512, 2) == ERR_WORKSPACE


def test_adapters(e4b):
    ws, bws = ctypes.c_size_t(0), ctypes.c_size_t(0)

    def fwd(**kw):
        kw.setdefault("groups", 1)
        return e4b._c_lora_ws(ctypes.byref(_forward(e4b, adapters=1, **kw)), ctypes.byref(ws))

    def bwd(**kw):
        kw.setdefault("groups", 1)
        return e4b._c_lora_bwd_ws(ctypes.byref(_backward(e4b, adapters=1, **kw)), ctypes.byref(bws))

    # long prefills of wide rows fit: their tiles are shared out over the columns as far as they are few
    assert fwd(S=1 << 23, K=4096, N=28672) == 0 and fwd(S=1 << 29, K=64, N=64) == 0
    assert fwd(S=1 << 30, K=64, N=64) == ERR_OVERFLOW  # 64 rows a workgroup
    # u: four lanes have four ranks of a row
    assert bwd(S=1 << 23, K=64, N=64) == 0
    assert bwd(S=1 << 30, K=64, N=64, r=128) == ERR_OVERFLOW
    assert e4b._c_lora_bwd(ctypes.byref(_backward(e4b, S=1 << 30, K=64, N=64, r=128, groups=1, adapters=1, ws_bytes=ROOM)),
                           None) == ERR_OVERFLOW
    # the adapters' gradients: 8192 elements a workgroup
    assert e4b._c_lora_bwd_ws(ctypes.byref(_backward(e4b, adapters=1 << 25, K=64, N=64)), ctypes.byref(bws)) == ERR_OVERFLOW


def test_binding_raises(e4b):
    with pytest.raises(e4b.E4BError, match="status -6"):
        e4b.e4b_permute_workspace_bytes(1 << 27, 512, 1)
