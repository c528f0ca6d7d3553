"""Refusals of the 8-bit row calls, the gated activation on rows, the MXFP4 rows and their product, before
any device is touched."""
import ctypes

import pytest
import torch

from test_lora_host import ERR_ALIGN, ERR_ARG, ERR_OVERFLOW, ERR_SHAPE, ERR_WORKSPACE, FAKE, _backward

BF16, F32, I8 = 0, 1, 2


def test_checkpoint_refuses(e4b):
    def f(x=FAKE, dtype=BF16, S=16, C=64, codes=FAKE, scales=FAKE):
        return e4b._c_checkpoint(x, dtype, S, C, codes, scales, None)
    assert f(dtype=I8) == ERR_ARG and f(dtype=-1) == ERR_ARG and f(S=-1) == ERR_ARG and f(C=0) == ERR_ARG
    assert f(x=None) == ERR_ARG and f(codes=None) == ERR_ARG and f(scales=None) == ERR_ARG
    assert f(C=48) == ERR_SHAPE
    assert f(x=FAKE + 8) == ERR_ALIGN and f(codes=FAKE + 8) == ERR_ALIGN and f(scales=FAKE + 1) == ERR_ALIGN
    # 8 bf16 or 4 float32 elements a lane, 2^32 lanes
    assert f(S=1 << 30, C=32) == ERR_OVERFLOW and f(dtype=F32, S=1 << 29, C=32) == ERR_OVERFLOW
    assert f(S=1 << 62, C=1 << 10) == ERR_OVERFLOW


def test_restore_refuses(e4b):
    def f(codes=FAKE, scales=FAKE, S=16, C=64, out=FAKE, dtype=BF16):
        return e4b._c_restore(codes, scales, S, C, out, dtype, None)
    assert f(dtype=I8) == ERR_ARG and f(S=-1) == ERR_ARG and f(C=-32) == ERR_ARG and f(C=33) == ERR_SHAPE
    assert f(codes=None) == ERR_ARG and f(scales=None) == ERR_ARG and f(out=None) == ERR_ARG
    assert f(out=FAKE + 4) == ERR_ALIGN and f(S=1 << 30, C=32) == ERR_OVERFLOW


def test_glu_refuses(e4b):
    def f(rows=FAKE, dtype=F32, rs=None, S=16, I=64, flags=0, h=FAKE, hdt=BF16, codes=None, scales=None):
        return e4b._c_glu(rows, dtype, rs, S, I, flags, h, hdt, codes, scales, None)
    assert f(dtype=3) == ERR_ARG and f(hdt=I8) == ERR_ARG and f(flags=1) == ERR_ARG and f(flags=0x40) == ERR_ARG
    assert f(S=-1) == ERR_ARG and f(I=0) == ERR_ARG and f(rows=None) == ERR_ARG and f(h=None) == ERR_ARG
    assert f(I=48) == ERR_SHAPE and f(I=24, flags=0x20) == ERR_SHAPE
    assert f(rs=FAKE) == ERR_ARG and f(dtype=I8) == ERR_ARG                  # scales with 8 bits, and only then
    assert f(codes=FAKE) == ERR_ARG and f(scales=FAKE) == ERR_ARG            # both or neither
    assert f(dtype=I8, rs=FAKE, codes=FAKE, scales=FAKE) == ERR_ARG
    assert f(rows=FAKE + 4) == ERR_ALIGN and f(h=FAKE + 2) == ERR_ALIGN and f(codes=FAKE + 8, scales=FAKE) == ERR_ALIGN
    assert f(S=1 << 29, I=32) == ERR_OVERFLOW


def test_glu_backward_refuses(e4b):
    def f(g=FAKE, gdt=BF16, rows=FAKE, dtype=I8, rs=FAKE, S=16, I=64, flags=0, out=FAKE, odt=BF16):
        return e4b._c_glu_bwd(g, gdt, rows, dtype, rs, S, I, flags, out, odt, None)
    assert f(gdt=I8) == ERR_ARG and f(odt=I8) == ERR_ARG and f(dtype=-1) == ERR_ARG and f(g=None) == ERR_ARG
    assert f(rs=None) == ERR_ARG and f(dtype=BF16) == ERR_ARG and f(out=None) == ERR_ARG
    assert f(I=40) == ERR_SHAPE and f(g=FAKE + 8) == ERR_ALIGN and f(rs=FAKE + 8) == ERR_ALIGN


def test_quantize_refuses(e4b):
    def f(x=FAKE, dtype=BF16, T=16, K=64, k=2, slots=FAKE, blocks=FAKE, scales=FAKE):
        return e4b._c_quant_mxfp4(x, dtype, T, K, k, slots, blocks, scales, None)
    assert f(dtype=I8) == ERR_ARG and f(T=-1) == ERR_ARG and f(K=0) == ERR_ARG and f(k=0) == ERR_ARG
    assert f(slots=None) == ERR_ARG                                          # k = 2 needs them
    assert f(x=None) == ERR_ARG and f(blocks=None) == ERR_ARG and f(scales=None) == ERR_ARG
    assert f(K=48) == ERR_SHAPE and f(k=65) == ERR_SHAPE
    assert f(x=FAKE + 8) == ERR_ALIGN and f(slots=FAKE + 4) == ERR_ALIGN and f(scales=FAKE + 2) == ERR_ALIGN
    assert f(T=1 << 30) == ERR_OVERFLOW and f(T=1 << 26, K=2048, k=1) == ERR_OVERFLOW


def _gemm(e4b, **kw):
    a = e4b.Mxfp4GemmArgs()
    a.E, a.N, a.K, a.S, a.out_dtype = 4, 64, 128, 100, F32
    for n in ("x", "x_scales", "w", "w_scales", "bias", "expert_offsets", "out"):
        setattr(a, n, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_product_refuses(e4b):
    f = lambda **kw: e4b._c_mxfp4_gemm(ctypes.byref(_gemm(e4b, **kw)), None)
    assert e4b._c_mxfp4_gemm(None, None) == ERR_ARG
    assert f(out_dtype=I8) == ERR_ARG and f(reserved=1) == ERR_ARG and f(E=0) == ERR_ARG and f(N=0) == ERR_ARG
    assert f(K=-32) == ERR_ARG and f(S=-1) == ERR_ARG and f(K=80) == ERR_SHAPE
    for n in ("x", "x_scales", "w", "w_scales", "expert_offsets", "out"):
        assert f(**{n: None}) == ERR_ARG, n
    for n in ("x", "x_scales", "w", "w_scales", "bias", "expert_offsets", "out"):
        assert f(**{n: FAKE + 8}) == ERR_ALIGN, n
    assert f(S=1 << 31) == ERR_OVERFLOW and f(K=1 << 24) == ERR_OVERFLOW and f(N=1 << 24) == ERR_OVERFLOW
    assert f(E=1 << 17) == ERR_OVERFLOW and f(S=(1 << 31) - 1, N=1 << 23) == ERR_OVERFLOW


def test_adapter_gradients_of_kept_rows_refuse(e4b):
    def f(codes=FAKE, scales=FAKE, **kw):
        kw.setdefault("x", None)
        return e4b._c_lora_bwd_x8(ctypes.byref(_backward(e4b, **kw)), codes, scales, None)
    assert f(x=FAKE) == ERR_ARG and f(codes=None) == ERR_ARG and f(scales=None) == ERR_ARG
    assert f(K=40) == ERR_SHAPE and f(codes=FAKE + 8) == ERR_ALIGN and f(scales=FAKE + 1) == ERR_ALIGN
    assert f(ws_bytes=0) == ERR_WORKSPACE and f(g=None) == ERR_ARG


def test_binding_refuses_host_tensors(e4b):
    x, q, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    w = torch.zeros(1, 8, 2, 16, dtype=torch.uint8)
    calls = (lambda: e4b.e4b_checkpoint_rows(x), lambda: e4b.e4b_restore_rows(q, s), lambda: e4b.e4b_glu(x),
             lambda: e4b.e4b_glu(q, s), lambda: e4b.e4b_glu_backward(x, q, s), lambda: e4b.e4b_quantize_act_mxfp4(x),
             lambda: e4b.e4b_grouped_gemm_mxfp4(w, s, w, s, s))
    for call in calls:
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        e4b.e4b_checkpoint_rows([1.0])
    with pytest.raises(ValueError, match="act must be"):
        e4b.e4b_glu(x, act="relu")


def test_empty_grids_need_no_device_buffers(e4b):
    """Without rows nothing is read or written: the pointers may be NULL (up to the device check)."""
    for st in (e4b._c_checkpoint(None, BF16, 0, 64, None, None, None), e4b._c_restore(None, None, 0, 64, None, BF16, None),
               e4b._c_glu(None, F32, None, 0, 64, 0, None, BF16, None, None, None),
               e4b._c_quant_mxfp4(None, BF16, 0, 64, 2, None, None, None, None),
               e4b._c_mxfp4_gemm(ctypes.byref(_gemm(e4b, S=0, x=None, out=None)), None)):
        assert st not in (ERR_ARG, ERR_ALIGN, ERR_SHAPE)
