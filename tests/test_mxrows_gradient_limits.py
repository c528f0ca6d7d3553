"""Where the MXFP4 product of rows and the dgrad that is its gradient part: the sizes that only the product takes are
refused by the dgrad, and over the scale bytes that both take the dgrad is the product's gradient."""
import ctypes

import pytest
import torch

import rows_reference as ref
from test_lora_host import ERR_ALIGN, ERR_ARG, ERR_OVERFLOW, ERR_SHAPE

REFUSED = (ERR_ALIGN, ERR_ARG, ERR_OVERFLOW, ERR_SHAPE)


@pytest.mark.parametrize("N,K,S,status", [(200, 128, 5, ERR_SHAPE), (64, 96, 5, ERR_SHAPE), (1, 32, 5, ERR_SHAPE), (64, 64, 5, 0),
                                          (1 << 16, 64, 1 << 15, ERR_OVERFLOW), (64, 1 << 16, 1 << 15, ERR_OVERFLOW),
                                          (1 << 16, 64, (1 << 15) - 1, 0), (1 << 16, 1 << 16, 5, ERR_OVERFLOW)])
def test_sizes(e4b, N, K, S, status):
    n = ctypes.c_size_t(0)
    assert e4b._c_dgrad_ws(ctypes.byref(e4b._dgrad_args("mxfp4", 4, N, K, S)), ctypes.byref(n)) == status
    a = e4b.Mxfp4GemmArgs()
    a.E, a.N, a.K, a.S, a.out_dtype = 4, N, K, 0, e4b.E4B_DT_F32  # without rows: the sizes' checks alone
    assert e4b._c_mxfp4_gemm(ctypes.byref(a), None) not in REFUSED


@pytest.mark.gpu
@pytest.mark.parametrize("low,high", [(104, 105), (140, 141), (104, 141)])
def test_gradient_over_the_scales_that_the_dgrad_takes(e4b, low, high):
    """<g, W x> = <W^T g, x> for every x: the dgrad against the transposed stack in float64.  Its weights and the
    gradients (halves up to 16) are fp16 values exactly, and their products float32 values; a float32 sum of
    N of them is off by (N + 2) 2^-24 of the sum of their magnitudes (two more for the order inside an instruction)."""
    from gpu_helpers import DEV
    E, N, K, S = 3, 192, 128, 70
    gen = torch.Generator(device=DEV)
    gen.manual_seed(low + high)
    w = torch.randint(0, 256, (E, N, K // 32, 16), dtype=torch.uint8, device=DEV, generator=gen)
    ws = torch.randint(low, high, (E, N, K // 32), dtype=torch.int32, device=DEV, generator=gen).to(torch.uint8)
    g = (torch.randint(-32, 33, (S, N), device=DEV, generator=gen) / 2).bfloat16()
    ends = [0, 33, 33, S]
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    out, _ = e4b.e4b_grouped_dgrad("mxfp4", g, w, ws, off)
    values = ref.mxfp4_values(w, ws)
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            want, mag = g[lo:hi].double() @ values[e], g[lo:hi].double().abs() @ values[e].abs()
            ref.assert_within(out[lo:hi], want, (N + 2) * 2.0 ** -24 * mag, f"expert {e}")
    # and the product's own rows against the same stack
    x4 = e4b.e4b_quantize_act_mxfp4(torch.randn(S, K, device=DEV, generator=gen))
    y, x = e4b.e4b_grouped_gemm_mxfp4(*x4, w, ws, off), ref.mxfp4_values(*x4)
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            want, mag = x[lo:hi] @ values[e].T.contiguous(), x[lo:hi].abs() @ values[e].abs().T.contiguous()
            ref.assert_within(y[lo:hi], want, (K + 2) * 2.0 ** -24 * mag, f"rows of expert {e}")
