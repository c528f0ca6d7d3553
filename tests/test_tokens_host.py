"""Refusals of the token permutation and combine calls, before any device is touched."""
import ctypes

import pytest
import torch

ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_OVERFLOW = -1, -2, -3, -4, -6
FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation first


def test_permute_refuses(e4b):
    def f(x=FAKE, dtype=0, T=16, H=64, k=2, slots=FAKE, rows=FAKE, ws=None, n=0):
        return e4b._c_permute(x, dtype, T, H, k, slots, rows, ws, n, None)
    assert f(dtype=2) == ERR_ARG and f(dtype=-1) == ERR_ARG
    assert f(T=-1) == ERR_ARG and f(H=0) == ERR_ARG and f(k=0) == ERR_ARG
    assert f(x=None) == ERR_ARG and f(slots=None) == ERR_ARG and f(rows=None) == ERR_ARG
    assert f(k=65) == ERR_SHAPE
    assert f(x=FAKE + 2) == ERR_ALIGN and f(rows=FAKE + 8) == ERR_ALIGN
    assert f(T=1 << 30, k=2) == ERR_OVERFLOW and f(H=1 << 31) == ERR_OVERFLOW
    need = e4b.e4b_permute_workspace_bytes(16384, 4096, 8)
    assert need >= 4 * 8 * 16384 and e4b.e4b_permute_workspace_bytes(16, 64, 2, torch.float32) == 0
    assert f(T=16384, H=4096, k=8) == ERR_WORKSPACE and f(T=16384, H=4096, k=8, ws=FAKE, n=need - 1) == ERR_WORKSPACE
    assert f(T=16384, H=4096, k=8, ws=FAKE + 4, n=need) == ERR_ALIGN
    assert f(T=1 << 62, k=64) == ERR_OVERFLOW and f(T=1 << 30, k=1, H=(1 << 31) - 1) == ERR_OVERFLOW


def test_combine_refuses(e4b):
    def f(rows=FAKE, rdt=1, T=16, H=64, k=2, slots=FAKE, w=FAKE, out=FAKE, odt=0, ws=None, n=0):
        return e4b._c_combine(rows, rdt, T, H, k, slots, w, out, odt, ws, n, None)
    assert f(rdt=2) == ERR_ARG and f(odt=9) == ERR_ARG
    assert f(rows=None) == ERR_ARG and f(out=None) == ERR_ARG and f(slots=None) == ERR_ARG
    assert f(w=FAKE + 4) == ERR_ALIGN and f(k=65) == ERR_SHAPE
    need = e4b.e4b_combine_workspace_bytes(4096, 4)
    assert need >= 4 * 4096 * 4 and e4b.e4b_combine_workspace_bytes(16, 2) == 0
    assert f(T=4096, k=4) == ERR_WORKSPACE
    assert f(T=4096, k=4, ws=FAKE, n=need - 1) == ERR_WORKSPACE


def test_combine_backward_refuses(e4b):
    def f(g=FAKE, gdt=0, rows=FAKE, rdt=1, T=16, H=64, k=2, slots=FAKE, w=FAKE, gr=FAKE, grdt=0, gw=FAKE, ws=None, n=0):
        return e4b._c_combine_bwd(g, gdt, rows, rdt, T, H, k, slots, w, gr, grdt, gw, ws, n, None)
    assert f(gdt=2) == ERR_ARG and f(rdt=3) == ERR_ARG and f(grdt=2) == ERR_ARG
    assert f(g=None) == ERR_ARG and f(w=None) == ERR_ARG and f(gr=None) == ERR_ARG
    assert f(rows=None) == ERR_ARG                       # g_w needs the rows
    assert f(gw=FAKE + 4) == ERR_ALIGN and f(T=8192) == ERR_WORKSPACE


def test_workspace_query_refuses(e4b):
    n = ctypes.c_size_t(0)
    assert e4b._c_combine_ws(16, 2, None) == ERR_ARG
    assert e4b._c_combine_ws(-1, 2, ctypes.byref(n)) == ERR_ARG
    assert e4b._c_combine_ws(1 << 31, 1, ctypes.byref(n)) == ERR_OVERFLOW
    with pytest.raises(e4b.E4BError):
        e4b.e4b_combine_workspace_bytes(4, 65)


def test_binding_refuses_host_tensors(e4b):
    x, slots = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: e4b.e4b_permute_tokens(x, slots, 2), lambda: e4b.e4b_combine_tokens(x, slots, 2),
                 lambda: e4b.e4b_combine_tokens_backward(x, None, slots, 2, torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        e4b.e4b_permute_tokens([1.0], slots, 2)
