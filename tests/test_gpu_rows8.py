"""Rows in 8 bits and the gated activation on rows with its gradient, against float64 (rows_reference.py
states the bounds)."""
import numpy as np
import pytest
import torch

import rows_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACTS = [("swiglu", False), ("swiglu", True), ("clamped_glu", False), ("clamped_glu", True)]


def _normal(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


def _bits(t):
    return t.view(torch.int16 if t.dtype == BF16 else torch.int32)


# ---- 8 bits


@pytest.mark.parametrize("S,C", [(1, 32), (1, 2880), (3, 96), (7, 64), (65, 2880), (1000, 1312), (4099, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_checkpoint_and_restore(e4b, S, C, dtype):
    x = _normal(S, C, dtype=dtype, seed=S, std=3.0) * torch.exp2(_normal(1, C, seed=1, std=4.0).round()).to(dtype)
    codes, scales = e4b.e4b_checkpoint_rows(x)
    q, s = ref.rows8_of(x)
    assert torch.equal(codes, q) and torch.equal(scales, s)
    for out in (BF16, F32):
        back = e4b.e4b_restore_rows(codes, scales, dtype=out)
        assert torch.equal(back.double(), ref.rows8_values(codes, scales))  # exact in both types
    # within half a step 2^(X - 7); the block's largest is at least 127.5 / 128 of 2^X, so that is 1 / 127.5 of it
    # at most (half a step against a largest of just 2^X is 2^-7, not the 2^-8 that a first form of this test had)
    err = (back.double() - x.double()).abs()
    assert (err <= torch.exp2(scales.double() - 134).repeat_interleave(32, -1)).all()
    top = x.double().abs().reshape(S, -1, 32).amax(-1).repeat_interleave(32, -1)
    assert (err <= top / 127.5).all()


def test_checkpoint_of_every_bf16_value(e4b):
    """Each of the 65536 bit patterns as the largest of a block of its own, beside zero and a half of it."""
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16)
    x = torch.zeros(65536, 32, dtype=BF16, device=DEV)
    x[:, 0] = bits.view(BF16)
    x[:, 7] = x[:, 0] / 2
    x[:, 31] = -x[:, 0] * 0.3
    codes, scales = e4b.e4b_checkpoint_rows(x)
    q, s = ref.rows8_of(x)
    assert torch.equal(scales, s) and torch.equal(codes, q)
    back = e4b.e4b_restore_rows(codes, scales)
    want = ref.rows8_values(codes, scales)
    bad = ~torch.isfinite(x).all(1)
    assert torch.isnan(back[bad]).all() and torch.equal(back[~bad].double(), want[~bad])


def test_checkpoint_at_the_ends_of_float32(e4b):
    top = torch.finfo(F32).max
    values = [0.0, 2.0 ** -149, 2.0 ** -133, 127.4 * 2.0 ** -133, 127.5 * 2.0 ** -133, 2.0 ** -126, 1.9921874, 1.9921875, 1.9999999,
              2.0, 2.0 ** 126 * 1.9999999, 2.0 ** 127, top, -top]
    x = torch.zeros(len(values), 64, device=DEV)
    x[:, 3] = torch.tensor(values, dtype=torch.float64).to(F32).to(DEV)
    x[:, 40] = 1.0
    codes, scales = e4b.e4b_checkpoint_rows(x)
    q, s = ref.rows8_of(x)
    assert torch.equal(codes, q) and torch.equal(scales, s)
    assert torch.equal(e4b.e4b_restore_rows(codes, scales, dtype=F32).double(), ref.rows8_values(q, s))


def test_blocks_that_are_not_finite_stay_among_themselves(e4b):
    x = _normal(5, 128, dtype=F32, seed=4)
    x[1, 40], x[2, 0], x[4, 127] = float("nan"), float("inf"), float("-inf")
    back = e4b.e4b_restore_rows(*e4b.e4b_checkpoint_rows(x), dtype=F32).reshape(5, 4, 32)
    bad = torch.zeros(5, 4, dtype=torch.bool, device=DEV)
    bad[1, 1] = bad[2, 0] = bad[4, 3] = True
    assert torch.isnan(back[bad]).all() and torch.isfinite(back[~bad]).all()


def test_rows_given_to_fill_and_no_others(e4b):
    x = _normal(33, 96, dtype=BF16, seed=5)
    codes = torch.full((35, 96), 55, dtype=torch.int8, device=DEV)
    scales = torch.full((35, 3), 99, dtype=torch.uint8, device=DEV)
    e4b.e4b_checkpoint_rows(x, codes[:33], scales[:33])
    q, s = ref.rows8_of(x)
    assert torch.equal(codes[:33], q) and torch.equal(scales[:33], s) and (codes[33:] == 55).all() and (scales[33:] == 99).all()
    out = torch.full((35, 96), 7.0, device=DEV)
    e4b.e4b_restore_rows(codes[:33], scales[:33], out=out[:33])
    assert torch.equal(out[:33].double(), ref.rows8_values(q, s)) and (out[33:] == 7).all()


# ---- the activation


SHAPES = [(1, 32), (1, 2880), (5, 96), (257, 2880), (1023, 160), (300, 1536)]


@pytest.mark.parametrize("S,I", SHAPES)
@pytest.mark.parametrize("act,interleaved", ACTS)
@pytest.mark.parametrize("rows_t", [BF16, F32, torch.int8])
@pytest.mark.parametrize("out_t", [BF16, F32])
def test_glu(e4b, S, I, act, interleaved, rows_t, out_t):
    rows = _normal(S, 2 * I, dtype=F32 if rows_t == torch.int8 else rows_t, seed=I, std=4.0)
    if rows_t == torch.int8:
        codes, scales = e4b.e4b_checkpoint_rows(rows)
        h, kept = e4b.e4b_glu(codes, scales, act=act, interleaved=interleaved, dtype=out_t)
        assert kept is None
        rows = ref.rows8_values(codes, scales)
    else:
        h, kept = e4b.e4b_glu(rows, act=act, interleaved=interleaved, dtype=out_t, checkpoint=True)
        q, s = ref.rows8_of(rows)
        assert torch.equal(kept[0], q) and torch.equal(kept[1], s)
        alone, none = e4b.e4b_glu(rows, act=act, interleaved=interleaved, dtype=out_t)
        assert none is None and torch.equal(alone, h)
    assert h.dtype == out_t
    ref.assert_within(h, *ref.glu(rows, act, interleaved), "h")


@pytest.mark.parametrize("S,I", SHAPES)
@pytest.mark.parametrize("act,interleaved", ACTS)
@pytest.mark.parametrize("rows_t", [BF16, F32, torch.int8])
@pytest.mark.parametrize("g_t,out_t", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_glu_backward(e4b, S, I, act, interleaved, rows_t, g_t, out_t):
    rows = _normal(S, 2 * I, dtype=F32 if rows_t == torch.int8 else rows_t, seed=I, std=4.0)
    g = _normal(S, I, dtype=g_t, seed=S + 1)
    given = (rows,)
    if rows_t == torch.int8:
        given = e4b.e4b_checkpoint_rows(rows)
        rows = ref.rows8_values(*given)
    d = e4b.e4b_glu_backward(g, *given, act=act, interleaved=interleaved, dtype=out_t)
    assert d.dtype == out_t and d.shape == (S, 2 * I)
    ref.assert_within(d, *ref.glu_backward(g, rows, act, interleaved), "g_rows")


def test_glu_of_sixteen_interleaved_pairs(e4b):
    rows = _normal(9, 32 * 3, seed=8, std=3.0)  # I = 48: not a multiple of 32
    h, kept = e4b.e4b_glu(rows, interleaved=True, dtype=F32, checkpoint=True)
    ref.assert_within(h, *ref.glu(rows, "swiglu", True), "h")
    d = e4b.e4b_glu_backward(_normal(9, 48, seed=9), *kept, interleaved=True, dtype=F32)
    ref.assert_within(d, *ref.glu_backward(_normal(9, 48, seed=9), ref.rows8_values(*kept), "swiglu", True), "g_rows")


@pytest.mark.parametrize("act,interleaved", ACTS)
def test_values_at_the_clamps_and_far_out(e4b, act, interleaved):
    v = torch.tensor([0.0, -0.0, 7.0, -7.0, 7.0000005, -7.0000005, 6.9999995, 1.702, -1.0, -1.278, 20.0, -20.0, 80.0, -80.0, 88.0, -88.0,
                      100.0, -100.0, 3e4, -3e4, 1e18, -1e18], device=DEV)
    n = len(v)
    gate, up = v.repeat_interleave(n), v.repeat(n)
    pad = (-len(gate)) % 32
    gate, up = (torch.cat([t, t[:pad]])[None] for t in (gate, up))
    rows = ref.joined(gate, up, interleaved).contiguous()
    ref.assert_within(e4b.e4b_glu(rows, act=act, interleaved=interleaved, dtype=F32)[0], *ref.glu(rows, act, interleaved), "h")
    g = torch.ones_like(gate)
    d = e4b.e4b_glu_backward(g, rows, act=act, interleaved=interleaved, dtype=F32)
    ref.assert_within(d, *ref.glu_backward(g, rows, act, interleaved), "g_rows")


@pytest.mark.parametrize("act,interleaved", ACTS)
def test_values_at_the_ends_of_float32(e4b, act, interleaved):
    """A gate far below zero shuts its pair, whatever the ups and gradients: the logistic function there is under
    2^-126 and counts as 0.  Far above zero it is 1."""
    top = torch.finfo(F32).max
    gate = torch.tensor([-top, -1e38, -1e30, -1e4, -200.0, -128.0, -105.0], device=DEV).repeat_interleave(32)[None]
    up = torch.tensor([top, -top, 1e38, 1.0, -1.0, 0.0, 7.0, -7.0], device=DEV).repeat(28)[None]
    g = torch.tensor([top, 1.0, -top, -1.0], device=DEV).repeat_interleave(8).repeat(7)[None]
    rows = ref.joined(gate, up, interleaved).contiguous()
    zero = torch.zeros_like(gate)
    assert torch.equal(e4b.e4b_glu(rows, act=act, interleaved=interleaved, dtype=F32)[0], zero)
    d = e4b.e4b_glu_backward(g, rows, act=act, interleaved=interleaved, dtype=F32)
    assert torch.equal(d, torch.zeros_like(d))
    high = ref.joined(-gate, torch.ones_like(gate), interleaved).contiguous()
    h = e4b.e4b_glu(high, act=act, interleaved=interleaved, dtype=F32)[0]
    d_gate, d_up = ref.halves(e4b.e4b_glu_backward(torch.ones_like(g), high, act=act, interleaved=interleaved, dtype=F32), interleaved)
    if act == "swiglu":
        assert torch.equal(h, -gate) and torch.equal(d_gate, torch.ones_like(gate)) and torch.equal(d_up, -gate)
    else:
        ref.assert_within(h, *ref.glu(high, act, interleaved), "h")
        assert torch.equal(d_gate, zero) and torch.equal(d_up, h / 2)


@pytest.mark.parametrize("act,interleaved", ACTS)
def test_gradient_against_differences(e4b, act, interleaved):
    """Central differences of the float64 forward with steps of 2^-10: a third derivative of a few units times
    step^2 / 6 is under 1e-5."""
    rows = _normal(64, 64, seed=11).clamp(-3, 3)
    g = _normal(64, 32, seed=12)
    d = ref.halves(e4b.e4b_glu_backward(g, rows, act=act, interleaved=interleaved, dtype=F32).double(), interleaved)
    gate, up = ref.halves(rows.double(), interleaved)
    for part, i in zip(d, (0, 1)):
        step = [2.0 ** -10 * (i == j) for j in (0, 1)]
        up_to, down_to = (ref.glu(ref.joined(gate + s * step[0], up + s * step[1], interleaved), act, interleaved)[0] for s in (1, -1))
        assert ((g.double() * (up_to - down_to) * 2.0 ** 9 - part).abs() <= 1e-5 * (1 + g.abs() * (1 + gate.abs()) * (1 + up.abs()))).all()


@pytest.mark.parametrize("act,interleaved", ACTS)
def test_nan_reaches_its_own_pair_alone(e4b, act, interleaved):
    gate, up = _normal(4, 64, seed=13), _normal(4, 64, seed=14)
    gate[1, 5], up[2, 60] = float("nan"), float("nan")
    rows = ref.joined(gate, up, interleaved).contiguous()
    bad = torch.isnan(gate) | torch.isnan(up)
    h = e4b.e4b_glu(rows, act=act, interleaved=interleaved, dtype=F32)[0]
    assert torch.equal(torch.isnan(h), bad)
    d_gate, d_up = ref.halves(e4b.e4b_glu_backward(torch.ones_like(gate), rows, act=act, interleaved=interleaved, dtype=F32), interleaved)
    assert not torch.isnan(d_gate[~bad]).any() and not torch.isnan(d_up[~bad]).any()
    assert torch.isnan(d_gate[1, 5]) and torch.isnan(d_gate[2, 60]) and torch.isnan(d_up[1, 5])


def test_no_rows(e4b):
    rows = torch.empty(0, 64, device=DEV)
    codes, scales = e4b.e4b_checkpoint_rows(rows)
    assert codes.shape == (0, 64) and scales.shape == (0, 2) and e4b.e4b_restore_rows(codes, scales).shape == (0, 64)
    h, kept = e4b.e4b_glu(rows, checkpoint=True)
    assert h.shape == (0, 32) and e4b.e4b_glu_backward(h, *kept).shape == (0, 64)


def test_refusals_of_the_binding(e4b):
    rows = _normal(4, 64, seed=15)
    codes, scales = e4b.e4b_checkpoint_rows(rows)
    with pytest.raises(ValueError, match="their own checkpoint"):
        e4b.e4b_glu(codes, scales, checkpoint=True)
    with pytest.raises(ValueError):
        e4b.e4b_glu(codes)                                             # 8 bits without scales
    with pytest.raises(ValueError):
        e4b.e4b_glu(rows, scales)                                      # scales without 8 bits
    with pytest.raises(ValueError):
        e4b.e4b_glu_backward(rows, rows)                               # g has the rows' width
    with pytest.raises(ValueError, match="contiguous"):
        e4b.e4b_checkpoint_rows(rows.t())
    with pytest.raises(ValueError):
        e4b.e4b_restore_rows(codes, scales[:3])
    with pytest.raises(e4b.E4BError):
        e4b.e4b_checkpoint_rows(_normal(4, 40))                        # not a multiple of 32
    with pytest.raises(e4b.E4BError):
        e4b.e4b_glu(_normal(4, 96))                                    # I = 48 in halves


def test_calls_on_another_stream_and_in_a_graph(e4b):
    rows, g = _normal(300, 2 * 1536, seed=16, std=2.0), _normal(300, 1536, dtype=BF16, seed=17)

    def step(stream=None):
        h, kept = e4b.e4b_glu(rows, checkpoint=True, stream=stream)
        return h, *kept, e4b.e4b_glu_backward(g, *kept, stream=stream), e4b.e4b_restore_rows(*kept, stream=stream)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(3):
        rows.copy_(_normal(300, 2 * 1536, seed=20 + i, std=2.0))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))
