"""Refusals of the adapter calls, before any device is touched."""
import ctypes

import pytest
import torch

ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_OVERFLOW = -1, -2, -3, -4, -6
FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation first


def _forward(e4b, **kw):
    a = e4b.LoraArgs()
    a.r, a.S, a.K, a.N, a.groups, a.adapters = 16, 100, 128, 64, 4, 4
    for n in ("x", "a", "b", "scale", "group_offsets", "group_adapter", "y", "out", "z", "ws"):
        setattr(a, n, FAKE)
    a.ws_bytes = 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _backward(e4b, **kw):
    a = e4b.LoraBackwardArgs()
    a.r, a.S, a.K, a.N, a.groups, a.adapters = 16, 100, 128, 64, 4, 4
    for n in ("g", "x", "z", "a", "b", "scale", "group_offsets", "group_adapter", "gx_base", "gx", "ga", "gb", "ws"):
        setattr(a, n, FAKE)
    a.ws_bytes = 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _check_sizes(f):
    assert f(S=-1) == ERR_ARG and f(K=0) == ERR_ARG and f(N=-8) == ERR_ARG and f(r=0) == ERR_ARG
    assert f(groups=0) == ERR_ARG and f(adapters=0) == ERR_ARG and f(reserved=1) == ERR_ARG
    assert f(r=12) == ERR_SHAPE and f(r=136) == ERR_SHAPE and f(K=100) == ERR_SHAPE and f(N=66) == ERR_SHAPE
    assert f(S=1 << 31) == ERR_OVERFLOW and f(adapters=1 << 31) == ERR_OVERFLOW and f(groups=1 << 31) == ERR_OVERFLOW
    assert f(S=1 << 30, N=1 << 30) == ERR_OVERFLOW and f(adapters=1 << 30, K=1 << 30) == ERR_OVERFLOW


def test_forward_refuses(e4b):
    f = lambda **kw: e4b._c_lora(ctypes.byref(_forward(e4b, **kw)), None)
    _check_sizes(f)
    assert f(out_dtype=2) == ERR_ARG
    for n in ("x", "a", "b", "group_offsets", "out", "ws"):
        assert f(**{n: None}) == ERR_ARG, n
    for n in ("x", "a", "b", "scale", "group_offsets", "group_adapter", "y", "out", "z", "ws"):
        assert f(**{n: FAKE + 8}) == ERR_ALIGN, n
    need = e4b.e4b_lora_workspace_bytes(100, 128, 64, 16, 4, 4)
    assert need >= 100 * 16 * 4 and f(ws_bytes=need - 1) == ERR_WORKSPACE
    assert e4b._c_lora(None, None) == ERR_ARG


def test_backward_refuses(e4b):
    f = lambda **kw: e4b._c_lora_bwd(ctypes.byref(_backward(e4b, **kw)), None)
    _check_sizes(f)
    assert f(gx_dtype=7) == ERR_ARG
    for n in ("g", "x", "z", "a", "b", "group_offsets", "ws"):
        assert f(**{n: None}) == ERR_ARG, n
    assert f(gx=None, ga=None, gb=None) == ERR_ARG
    for n in ("g", "x", "z", "a", "b", "scale", "gx_base", "gx", "ga", "gb", "ws"):
        assert f(**{n: FAKE + 4}) == ERR_ALIGN, n
    need = e4b.e4b_lora_backward_workspace_bytes(100, 128, 64, 16, 4, 4, group_adapter=True)
    assert f(ws_bytes=need - 1) == ERR_WORKSPACE
    assert e4b.e4b_lora_backward_workspace_bytes(100, 128, 64, 16, 4, 4, gx=False, ga=False) < need


def test_workspace_queries_refuse(e4b):
    n = ctypes.c_size_t(0)
    assert e4b._c_lora_ws(ctypes.byref(_forward(e4b)), None) == ERR_ARG
    assert e4b._c_lora_bwd_ws(None, ctypes.byref(n)) == ERR_ARG
    for bad in (dict(r=12), dict(K=4), dict(adapters=0)):
        size = dict(S=8, K=64, N=64, r=8, groups=1, adapters=1)
        size.update(bad)
        with pytest.raises(e4b.E4BError):
            e4b.e4b_lora_workspace_bytes(**size)
        with pytest.raises(e4b.E4BError):
            e4b.e4b_lora_backward_workspace_bytes(**size)


def test_empty_batch_needs_no_rows(e4b):
    assert e4b.e4b_lora_workspace_bytes(0, 64, 64, 8, 3, 3) >= 0
    assert e4b.e4b_lora_backward_workspace_bytes(0, 64, 64, 8, 3, 3) >= 0


def test_binding_refuses_host_tensors(e4b):
    x, a, b = torch.zeros(4, 16), torch.zeros(1, 8, 16), torch.zeros(1, 24, 8)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        e4b.e4b_grouped_lora(x, a, b, None, off)
    with pytest.raises(ValueError, match="device tensor"):
        e4b.e4b_grouped_lora_backward(torch.zeros(4, 24), x, None, a, b, None, off)
