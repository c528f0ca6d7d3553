"""The MXFP4 rows, their products, the activation and the 8-bit rows together, as a training step and a decode
step of the expert layer make them: each call's result against float64 from what the call was given."""
import pytest
import torch

import rows_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _normal(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


def _stack(e4b, E, N, K, seed):
    return e4b.e4b_pack_mxfp4(_normal(E, N, K, dtype=BF16, seed=seed, std=K ** -0.5))


def _check_product(out, x4, w4, off, bias):
    x, w, K = ref.mxfp4_values(*x4), ref.mxfp4_values(*w4), x4[1].shape[1] * 32
    for e in range(w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            want, mag = x[lo:hi] @ w[e].T.contiguous(), x[lo:hi].abs() @ w[e].abs().T.contiguous()
            if bias is not None:
                want, mag = want + bias[e].double(), mag + bias[e].double().abs()
            ref.assert_within(out[lo:hi], want, (K + 2) * 2.0 ** -24 * mag, f"rows of expert {e}")


@pytest.mark.parametrize("act,interleaved", [("swiglu", False), ("clamped_glu", True)])
@pytest.mark.parametrize("T,E,k,H,I,r", [(96, 8, 2, 256, 192, 16), (300, 5, 3, 320, 448, 32)])
def test_training_step(e4b, act, interleaved, T, E, k, H, I, r):
    x = _normal(T, H, dtype=BF16, seed=1)
    _, w, off, slots = e4b.e4b_route_permute(_normal(T, E, seed=2), k)
    gu4, dn4 = _stack(e4b, E, 2 * I, H, 3), _stack(e4b, E, H, I, 4)
    b_gu = _normal(E, 2 * I, seed=5, std=0.1)
    a1, b1 = _normal(E, r, H, dtype=BF16, seed=6, std=H ** -0.5), _normal(E, 2 * I, r, dtype=BF16, seed=7, std=0.1)
    a2, b2 = _normal(E, r, I, dtype=BF16, seed=8, std=I ** -0.5), _normal(E, H, r, dtype=BF16, seed=9, std=0.1)
    scale = torch.full((E,), 2.0, device=DEV)
    form = {"act": act, "interleaved": interleaved}

    # forward
    x4 = e4b.e4b_quantize_act_mxfp4(x, slots, k)
    gu = e4b.e4b_grouped_gemm_mxfp4(*x4, *gu4, off, bias=b_gu)
    _check_product(gu, x4, gu4, off, b_gu)
    rows = e4b.e4b_permute_tokens(x, slots, k)
    gu, z1 = e4b.e4b_grouped_lora(rows, a1, b1, scale, off, y=gu, out=gu, z=True)
    h, kept = e4b.e4b_glu(gu, checkpoint=True, **form)
    ref.assert_within(h, *ref.glu(gu, act, interleaved), "h")
    codes, scales = ref.rows8_of(gu)
    assert torch.equal(kept[0], codes) and torch.equal(kept[1], scales)
    h4 = e4b.e4b_quantize_act_mxfp4(h)
    y = e4b.e4b_grouped_gemm_mxfp4(*h4, *dn4, off)
    _check_product(y, h4, dn4, off, None)
    y, z2 = e4b.e4b_grouped_lora(h, a2, b2, scale, off, y=y, out=y, z=True)
    out = e4b.e4b_combine_tokens(y, slots, k, w)
    rows8, h8 = e4b.e4b_checkpoint_rows(rows), e4b.e4b_checkpoint_rows(h)

    # backward: nothing of the forward's rows but the 8-bit ones, z and y
    g_out = _normal(T, H, dtype=BF16, seed=10)
    g_y, g_w = e4b.e4b_combine_tokens_backward(g_out, y, slots, k, w)
    g_h, _ = e4b.e4b_grouped_dgrad("mxfp4", g_y, *dn4, off)
    base_h = g_h.clone()
    g_h, ga2, gb2 = e4b.e4b_grouped_lora_backward(g_y, h8[0], z2, a2, b2, scale, off, gx_base=g_h, gx=g_h, x_scales=h8[1])
    g_gu = e4b.e4b_glu_backward(g_h, *kept, **form)
    ref.assert_within(g_gu, *ref.glu_backward(g_h, ref.rows8_values(*kept), act, interleaved), "g_gu")
    g_rows, _ = e4b.e4b_grouped_dgrad("mxfp4", g_gu, *gu4, off)
    base_r = g_rows.clone()
    g_rows, ga1, gb1 = e4b.e4b_grouped_lora_backward(g_gu, rows8[0], z1, a1, b1, scale, off, gx_base=g_rows, gx=g_rows, x_scales=rows8[1])
    g_x = e4b.e4b_combine_tokens(g_rows, slots, k)

    # the adapters' gradients: from the restored rows, and the formula
    same = e4b.e4b_grouped_lora_backward(g_gu, e4b.e4b_restore_rows(*rows8), z1, a1, b1, scale, off, gx_base=base_r)
    assert torch.equal(same[0], g_rows) and torch.equal(same[1], ga1) and torch.equal(same[2], gb1)
    same = e4b.e4b_grouped_lora_backward(g_y, e4b.e4b_restore_rows(*h8), z2, a2, b2, scale, off, gx_base=base_h)
    assert torch.equal(same[0], g_h) and torch.equal(same[1], ga2) and torch.equal(same[2], gb2)
    for ga, g, b, kept8 in ((ga1, g_gu, b1, rows8), (ga2, g_y, b2, h8)):
        xv = ref.rows8_values(*kept8)
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            u = 2.0 * (g[lo:hi].double() @ b[e].double())
            mag = 2.0 * (g[lo:hi].double().abs() @ b[e].double().abs())
            n = g.shape[1] + (hi - lo) + 8  # sums of u over the columns and of the gradient over the rows
            want, bound = u.T @ xv[lo:hi], n * 2.0 ** -24 * (mag.T @ xv[lo:hi].abs())
            ref.assert_within(ga[e], want, bound + 1e-30, f"adapter {e}")
    assert out.shape == g_x.shape == (T, H) and torch.isfinite(out).all() and torch.isfinite(g_x).all()
    assert g_w.shape == (T, k)


def test_decode_step_in_a_graph(e4b):
    """Four tokens through both products, captured and replayed on new tokens."""
    T, E, k, H, I = 4, 16, 4, 512, 384
    x, logits = _normal(T, H, dtype=BF16, seed=1), _normal(T, E, seed=2)
    gu4, dn4 = _stack(e4b, E, 2 * I, H, 3), _stack(e4b, E, H, I, 4)

    def step():
        _, w, off, slots = e4b.e4b_route_permute(logits, k)
        gu = e4b.e4b_grouped_gemm_mxfp4(*e4b.e4b_quantize_act_mxfp4(x, slots, k), *gu4, off)
        h, _ = e4b.e4b_glu(gu)
        return e4b.e4b_combine_tokens(e4b.e4b_grouped_gemm_mxfp4(*e4b.e4b_quantize_act_mxfp4(h), *dn4, off), slots, k, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(_normal(T, H, dtype=BF16, seed=20 + i))
        logits.copy_(_normal(T, E, seed=30 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())


def test_two_streams_at_once(e4b):
    """The calls have no workspace of their own: two streams run them side by side."""
    w4 = _stack(e4b, 8, 512, 1024, 3)
    off = torch.arange(0, 8 * 40 + 1, 40, dtype=torch.int32, device=DEV)
    xs = [_normal(320, 1024, dtype=BF16, seed=s) for s in (1, 2)]
    step = lambda x, s=None: e4b.e4b_glu(e4b.e4b_grouped_gemm_mxfp4(*e4b.e4b_quantize_act_mxfp4(x, stream=s), *w4, off, stream=s), stream=s)[0]
    want = [step(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[step(x, s) for _ in range(5)] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for gs, w in zip(got, want) for g in gs)
