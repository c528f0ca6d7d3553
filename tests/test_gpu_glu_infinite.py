"""The gated activation and its gradient where a gate or an up is infinite or NaN: which results are NaN, infinite or 0
as the calls state it, and the finite ones beside them against float64."""
import math

import pytest
import torch

import rows_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan
GATES = [-INF, -200.0, -1.0, 0.0, 2.0, 7.0, 9.0, INF, NAN]
UPS = [-INF, -9.0, -7.0, -1.0, 0.0, 3.0, 7.0, INF, NAN]
GRADS = [1.0, -0.5, 0.0]
ACTS = [("swiglu", False), ("swiglu", True), ("clamped_glu", False), ("clamped_glu", True)]


def _inputs():
    """Every gate with every up and every gradient, one after the other, the last block filled up with the first ones."""
    grid = torch.cartesian_prod(*(torch.tensor(v, dtype=torch.float64) for v in (GATES, UPS, GRADS)))
    n = -(-len(grid) // 32) * 32
    return grid[torch.arange(n) % len(grid)].T[:, None].unbind(0)


def _parts(gate, up, act):
    """The gate, the up's factor, t, and the logistic function of t and of -t, 0 below 2^-126."""
    if act == "swiglu":
        a, b, t = gate, up, gate
    else:
        a, b = torch.where(gate > 7, 7.0, gate), torch.where(up > 7, 7.0, torch.where(up < -7, -7.0, up)) + 1
        t = 1.702 * a
    s, rest = torch.sigmoid(t), torch.sigmoid(-t)
    return a, b, t, torch.where(s < 2.0 ** -126, 0.0, s), torch.where(rest < 2.0 ** -126, 0.0, rest)


def _same(got, want, bound, what):
    """NaN and infinities in the same places, what is finite within the bound."""
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]) and torch.equal(torch.isinf(got), inf), what
    fine = torch.isfinite(want)
    assert ((got - want).abs()[fine] <= bound[fine]).all(), what


def _bound(t, size, out_t):
    """rows_reference's: a float32 value off by its relative error or what is below 2^-126, rounded once."""
    return (2 * ref._rel(t.nan_to_num(nan=0.0)) + 1.001 * ref.HALF_STEP[out_t]) * size + 2.0 ** -120


@pytest.mark.parametrize("act,interleaved", ACTS)
@pytest.mark.parametrize("rows_t", [BF16, F32])
@pytest.mark.parametrize("out_t", [BF16, F32])
def test_forward(e4b, act, interleaved, rows_t, out_t):
    gate, up, _ = _inputs()
    rows = ref.joined(gate, up, interleaved).to(rows_t).to(DEV).contiguous()
    a, b, t, s, _ = _parts(gate, up, act)
    want = a * s * b
    h, _ = e4b.e4b_glu(rows, act=act, interleaved=interleaved, dtype=out_t)
    _same(h, want, _bound(t, want.abs(), out_t), "h")
    assert torch.isnan(want[gate == -INF]).all()  # in both forms, as torch's silu has it


@pytest.mark.parametrize("act,interleaved", ACTS)
@pytest.mark.parametrize("rows_t", [BF16, F32])
@pytest.mark.parametrize("out_t", [BF16, F32])
def test_backward(e4b, act, interleaved, rows_t, out_t):
    gate, up, g = _inputs()
    rows = ref.joined(gate, up, interleaved).to(rows_t).to(DEV).contiguous()
    a, b, t, s, rest = _parts(gate, up, act)
    factor = s * (1 + t * rest)
    if act == "clamped_glu":
        factor = torch.where(gate == -INF, 0.0, factor)
    d_gate, d_up = factor * b * g, a * s * g
    if act == "clamped_glu":
        d_gate, d_up = torch.where(gate > 7, 0.0, d_gate), torch.where(up.abs() > 7, 0.0, d_up)
    e_gate = _bound(t, (s * b * g).abs() * (1 + (t * rest).abs()), out_t)
    e_up = _bound(t, d_up.abs(), out_t)
    d = e4b.e4b_glu_backward(g.to(F32).to(DEV), rows, act=act, interleaved=interleaved, dtype=out_t)
    got = ref.halves(d, interleaved)
    _same(got[0], d_gate, e_gate.nan_to_num(nan=2.0 ** -120, posinf=2.0 ** -120), "g_gate")
    _same(got[1], d_up, e_up, "g_up")


@pytest.mark.parametrize("act,interleaved", ACTS)
def test_pairs_of_a_block_that_was_not_finite(e4b, act, interleaved):
    """From 8 bits a block with an infinity is all NaN: so is what is computed from it, and no other block's."""
    gate, up = torch.ones(1, 96), torch.full((1, 96), 2.0)
    gate[0, 40] = -INF
    rows = ref.joined(gate, up, interleaved).to(DEV).contiguous()
    _, kept = e4b.e4b_glu(rows, act=act, interleaved=interleaved, checkpoint=True)
    h, _ = e4b.e4b_glu(*kept, act=act, interleaved=interleaved, dtype=F32)
    bad_gate, bad_up = ref.halves(torch.isnan(ref.rows8_values(*kept)), interleaved)
    assert bad_gate[0, 40] and 0 < int((bad_gate | bad_up).sum()) <= 32 and torch.equal(torch.isnan(h), bad_gate | bad_up)
    d = e4b.e4b_glu_backward(torch.ones(1, 96, device=DEV), *kept, act=act, interleaved=interleaved, dtype=F32)
    d_gate, d_up = ref.halves(torch.isnan(d), interleaved)
    assert torch.equal(d_gate, bad_gate | bad_up) and torch.equal(d_up, bad_gate)
