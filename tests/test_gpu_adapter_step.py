"""The calls together, as a program makes them: a decode step with adapters beside the routed int4
projection, and a training step of adapters beside a frozen NF4 projection whose input gradient is
e4b_grouped_dgrad."""
import numpy as np
import pytest
import torch

from gpu_helpers import DEV, dev_bf16, host
from moe_inputs import f32_to_bf16_bits
from oracle import nf4 as onf4

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
E24 = 2.0 ** -23  # an addition of the matrix unit, whichever way it rounds


def _normal(seed, *shape, dtype=BF16, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


def _adapters(n, r, K, N, seed):
    scale = torch.rand(n, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)) + 0.5
    return _normal(seed + 1, n, r, K, std=K ** -0.5), _normal(seed + 2, n, N, r, std=r ** -0.5), scale


def _experts(offsets):
    o = host(offsets)
    return [(e, slice(int(o[e]), int(o[e + 1]))) for e in range(len(o) - 1) if o[e + 1] > o[e]]


@pytest.mark.parametrize("T", [1, 7, 64])
def test_decode_step_with_adapters_beside_the_int4_projection(e4b, T):
    """route -> gather -> routed int4 GEMV -> each expert's adapter in place -> combine, eager and as one
    captured graph replayed over changing tokens."""
    E, K, N, k, r = 16, 512, 256, 4, 16
    rng = np.random.default_rng(T)
    w = f32_to_bf16_bits((0.02 * rng.standard_normal((E, N, K))).astype(np.float32))
    packed, scales = e4b.e4b_pack_int4_b32(dev_bf16(w))
    a, b, scale = _adapters(E, r, K, N, 100 + T)
    x, logits = _normal(1, T, K), _normal(2, T, E, dtype=F32)

    def step():
        _, tw, off, slots = e4b.e4b_route_permute(logits, k)
        rows = e4b.e4b_permute_tokens(x, slots, k)
        y = e4b.e4b_gemv_int4_b32(packed, scales, x, k, off, slots)
        base = y.clone()
        e4b.e4b_grouped_lora(rows, a, b, scale, off, y=y, out=y)
        return tw, off, slots, base, e4b.e4b_combine_tokens(y, slots, k, tw, dtype=F32)

    tw, off, slots, base, out = step()
    s = slots.long()
    rows = x.double()[s // k]
    y, mag = base.double(), base.double().abs()
    for e, p in _experts(off):
        z = rows[p] @ a[e].double().T
        y[p] += scale[e].double() * (z @ b[e].double().T)
        zm = rows[p].abs() @ a[e].double().abs().T
        mag[p] += scale[e].double() * (zm @ b[e].double().abs().T)
    wd = tw.double().reshape(-1)[s, None]
    ref, bound = torch.zeros(T, N, dtype=torch.float64, device=DEV), torch.zeros(T, N, dtype=torch.float64, device=DEV)
    ref.index_add_(0, s // k, wd * y)
    # K + 3 r + a few roundings of the adapter, k of the combine, each of the magnitudes' sum
    bound.index_add_(0, s // k, wd * mag * ((K + 3 * r + k + 10) * E24))
    assert torch.isfinite(out).all() and ((out.double() - ref).abs() <= bound).all()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(3):
        x.copy_(_normal(10 + i, T, K))
        logits.copy_(_normal(20 + i, T, E, dtype=F32))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(captured, step())), i


def test_training_step_of_adapters_beside_a_frozen_nf4_projection(e4b):
    """out = combine(w, rows W^T + adapter): all gradients of <g, out> from the calls, against the
    formula in float64 on the decoded weights."""
    T, E, K, N, k, r = 150, 6, 256, 320, 2, 16
    rng = np.random.default_rng(3)
    wbits = f32_to_bf16_bits((0.05 * rng.standard_normal((E, N, K))).astype(np.float32))
    packed, absmax = e4b.e4b_pack_nf4(dev_bf16(wbits))
    W = torch.from_numpy(np.stack([onf4.dequantize(host(packed)[e], host(absmax)[e]) for e in range(E)])).double().to(DEV)
    a, b, scale = _adapters(E, r, K, N, 7)
    x, g = _normal(1, T, K), _normal(2, T, N)
    _, tw, off, slots = e4b.e4b_route_permute(_normal(3, T, E, dtype=F32), k)
    s = slots.long()

    # forward: the frozen projection's rows are made here (its gradient below is the framework's)
    rows = e4b.e4b_permute_tokens(x, slots, k)
    y = torch.empty(T * k, N, device=DEV)
    for e, p in _experts(off):
        y[p] = (rows[p].double() @ W[e].T).float()
    y, z = e4b.e4b_grouped_lora(rows, a, b, scale, off, y=y, z=True)
    out = e4b.e4b_combine_tokens(y, slots, k, tw, dtype=F32)
    # backward
    gy, gw = e4b.e4b_combine_tokens_backward(g, y, slots, k, tw)
    base, _ = e4b.e4b_grouped_dgrad("nf4", gy, packed, absmax, off)
    grows, ga, gb = e4b.e4b_grouped_lora_backward(gy, rows, z, a, b, scale, off, gx_base=base)
    gx = e4b.e4b_combine_tokens(grows, slots, k, dtype=F32)

    # the formula, on the bf16 gradient rows that the calls hand on
    wd = tw.double().reshape(-1)[s, None]
    gyd = (g.double()[s // k] * wd)
    assert ((gy.double() - gyd).abs() <= 2.0 ** -8 * 1.001 * gyd.abs()).all()
    gyd = gy.double()
    rd, rgx = rows.double(), torch.zeros(T * k, K, dtype=torch.float64, device=DEV)
    rga, rgb = torch.zeros_like(a, dtype=torch.float64), torch.zeros_like(b, dtype=torch.float64)
    for e, p in _experts(off):
        u = scale[e].double() * (gyd[p] @ b[e].double())
        rgx[p] = gyd[p] @ W[e] + u @ a[e].double()
        rga[e] = u.T @ rd[p]
        rgb[e] = scale[e].double() * (gyd[p].T @ (rd[p] @ a[e].double().T))
    rx = torch.zeros(T, K, dtype=torch.float64, device=DEV).index_add_(0, s // k, rgx)
    # dgrad decodes to fp16 weights (two roundings of 2^-11 each, averaging over N terms): its own
    # bound on a row, 8e-3 of the row's rms + 1e-3, covers gx's k rows; ga and gb are float32 sums
    tol = k * (8e-3 * rgx.square().mean(1).sqrt().max() + 1e-3)
    assert torch.isfinite(gx).all() and float((gx.double() - rx).abs().max()) <= float(tol)
    for got, ref in ((ga, rga), (gb, rgb)):
        assert float((got.double() - ref).norm() / ref.norm()) <= (N + K) * E24
    ref_w = (g.double()[s // k] * y.double()).sum(1)
    mag_w = (g.double()[s // k] * y.double()).abs().sum(1)
    assert ((gw.double().reshape(-1)[s] - ref_w).abs() <= (N + 1) * 2.0 ** -24 * mag_w).all()

    # and against differences: the change of <g, out> under a change of B alone is <gb, change> up to
    # gb's roundings of the gradient rows to bf16 (2^-8 of each product)
    b2 = (b.float() + _normal(9, *b.shape, dtype=F32, std=0.1)).to(BF16)
    y2, _ = e4b.e4b_grouped_lora(rows, a, b2, scale, off, y=y)
    y1, _ = e4b.e4b_grouped_lora(rows, a, b, scale, off, y=y)
    change = e4b.e4b_combine_tokens(y2, slots, k, tw, dtype=F32).double() - e4b.e4b_combine_tokens(y1, slots, k, tw, dtype=F32).double()
    left = float((g.double() * change).sum())
    step = b2.double() - b.double()
    right = float((gb.double() * step).sum())
    size = sum(float((scale[e].double() * (gyd[p].abs().T @ z[p].double().abs()) * step[e].abs()).sum())
               for e, p in _experts(off))
    # the float32 roundings: of y1 and y2 (a few steps of their magnitude, weighted by |g|) and of the sums
    ymag = float((gyd.abs() * y.double().abs()).sum())
    assert abs(left - right) <= 1.001 * 2.0 ** -8 * size + (3 * r + k + 8) * E24 * 4 * ymag
    assert out.shape == (T, N)
