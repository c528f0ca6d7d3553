"""Rows and stacks past 2^31 elements and 2^32 bytes: the first, a middle and the last rows against float64."""
import pytest
import torch

import rows_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _normal(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g, dtype=dtype) * std


def _some(S):
    return [slice(0, 3), slice(S // 2, S // 2 + 3), slice(S - 3, S)]


def test_rows_in_8_bits(e4b):
    S, C = 70001, 32768  # 2.3e9 elements, 4.6 GB of bf16
    x = _normal(S, C, dtype=BF16, seed=1)
    codes, scales = e4b.e4b_checkpoint_rows(x)
    back = e4b.e4b_restore_rows(codes, scales)
    for rows in _some(S):
        q, s = ref.rows8_of(x[rows])
        assert torch.equal(codes[rows], q) and torch.equal(scales[rows], s)
        assert torch.equal(back[rows].double(), ref.rows8_values(q, s))


@pytest.mark.parametrize("interleaved", [False, True])
def test_activation(e4b, interleaved):
    S, I = 40003, 28672  # 2.3e9 elements of rows
    rows, g = _normal(S, 2 * I, dtype=BF16, seed=2, std=2.0), _normal(S, I, dtype=BF16, seed=3)
    h, kept = e4b.e4b_glu(rows, interleaved=interleaved, checkpoint=True)
    d = e4b.e4b_glu_backward(g, *kept, interleaved=interleaved)
    for part in _some(S):
        ref.assert_within(h[part], *ref.glu(rows[part], "swiglu", interleaved), "h")
        values = ref.rows8_values(kept[0][part], kept[1][part])
        ref.assert_within(d[part], *ref.glu_backward(g[part], values, "swiglu", interleaved), "g_rows")


def _check_rows(out, x4, w4, expert, rows):
    x, w = ref.mxfp4_values(x4[0][rows], x4[1][rows]), ref.mxfp4_values(w4[0][expert], w4[1][expert])
    K = x.shape[1]
    ref.assert_within(out[rows], x @ w.T.contiguous(), (K + 2) * 2.0 ** -24 * (x.abs() @ w.abs().T.contiguous()), "rows")


def test_product_with_many_outputs(e4b):
    S, N, K = 40003, 60000, 64  # 2.4e9 outputs
    x4 = e4b.e4b_quantize_act_mxfp4(_normal(S, K, seed=4))
    w4 = e4b.e4b_pack_mxfp4(_normal(1, N, K, dtype=BF16, seed=5))
    off = torch.tensor([0, S], dtype=torch.int32, device=DEV)
    out = e4b.e4b_grouped_gemm_mxfp4(*x4, *w4, off, dtype=BF16)
    for rows in _some(S):
        _check_rows(out, x4, w4, 0, rows)


def test_product_with_a_stack_past_four_gigabytes(e4b):
    E, N, K, S = 40, 57344, 4096, 200  # 4.7 GB of codes
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    w4 = (torch.randint(0, 256, (E, N, K // 32, 16), dtype=torch.uint8, device=DEV, generator=g),
          torch.randint(100, 140, (E, N, K // 32), dtype=torch.uint8, device=DEV, generator=g))
    x4 = e4b.e4b_quantize_act_mxfp4(_normal(S, K, seed=7))
    off = torch.arange(0, S + 1, S // E, dtype=torch.int32, device=DEV)
    out = e4b.e4b_grouped_gemm_mxfp4(*x4, *w4, off)
    for e in (0, E // 2, E - 1):
        _check_rows(out, x4, w4, e, slice(5 * e, 5 * e + 5))


def test_gather_of_many_rows(e4b):
    T, K, k = 150001, 4096, 4  # 2.5e9 elements of rows
    x = _normal(T, K, dtype=BF16, seed=8)
    slots = torch.randperm(T * k, device=DEV).int()
    blocks, scales = e4b.e4b_quantize_act_mxfp4(x, slots, k)
    for rows in _some(T * k):
        b, s = e4b.e4b_quantize_act_mxfp4(x[slots[rows].long() // k].contiguous())
        assert torch.equal(blocks[rows], b) and torch.equal(scales[rows], s)


def test_many_experts(e4b):
    """More experts than a wave has lanes, most of them empty, as many as are taken."""
    for E in (65, 700, 65536):
        N, K, S = 40, 64, 90
        w4 = e4b.e4b_pack_mxfp4(_normal(E, N, K, dtype=BF16, seed=9))
        x4 = e4b.e4b_quantize_act_mxfp4(_normal(S, K, seed=10))
        of = torch.sort(torch.randint(0, E, (S,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(E)))[0]
        off = torch.searchsorted(of, torch.arange(E + 1, device=DEV)).int()
        out = e4b.e4b_grouped_gemm_mxfp4(*x4, *w4, off)
        x, w = ref.mxfp4_values(*x4), ref.mxfp4_values(*w4)[of]
        want, mag = torch.bmm(w, x[:, :, None])[..., 0], torch.bmm(w.abs(), x.abs()[:, :, None])[..., 0]
        ref.assert_within(out, want, (K + 2) * 2.0 ** -24 * mag, f"{E} experts")
