"""Float64 references of the row calls: MXFP4 and 8-bit values, the gated activation and its gradient."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def mxfp4_values(blocks, scales):
    """float64 values [.., K] of e2m1 codes [.., K/32, 16] and e8m0 bytes [.., K/32]; byte 255 is NaN."""
    code = torch.stack([blocks & 15, blocks >> 4], -1).flatten(-2).long()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=blocks.device)
    v = grid[code & 7] * torch.where(code >= 8, -1.0, 1.0).double()
    s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127))
    return (v * s[..., None]).flatten(-2)


def rows8_of(x):
    """(codes, scales) of the 8-bit checkpoint's definition, in float64."""
    v = x.double().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(v).all(-1)
    v = torch.where(bad[..., None], torch.zeros_like(v), v)
    top = v.abs().amax(-1)
    X = torch.where(top > 0, torch.floor(torch.log2(top.clamp_min(1e-60))), torch.full_like(top, -127.0)).clamp_min(-127)
    X = torch.where((torch.round(top * torch.exp2(6 - X)) >= 128) & (X < 127), X + 1, X)
    q = torch.round(v * torch.exp2(6 - X)[..., None]).clamp(-127, 127)
    byte = torch.where(bad, 255.0, X + 127)
    return q.reshape(x.shape).to(torch.int8), byte.to(torch.uint8)


def rows8_values(codes, scales):
    s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 133))
    return codes.double() * s.repeat_interleave(32, -1)


def halves(rows, interleaved):
    I = rows.shape[1] // 2
    return (rows[:, 0::2], rows[:, 1::2]) if interleaved else (rows[:, :I], rows[:, I:])


def joined(gate, up, interleaved):
    return torch.stack([gate, up], -1).flatten(-2) if interleaved else torch.cat([gate, up], -1)


def _parts(rows, act, interleaved):
    gate, up = halves(rows.double(), interleaved)
    if act == "swiglu":
        return gate, up, gate, up, gate, torch.ones_like(gate, dtype=torch.bool), torch.ones_like(up, dtype=torch.bool)
    gc, uc = gate.clamp(max=7.0), up.clamp(-7.0, 7.0)
    return gate, up, gc, uc + 1.0, 1.702 * gc, gate <= 7.0, up.abs() <= 7.0


# The kernels take e = 2^(t log2 e) and 1 / (1 + e) from the hardware.  t (a product for the clamped form, with a
# rounded constant), its product with a rounded log2 e: at most 4 |t| 2^-24 relative in e; the two
# instructions an ulp each, the sum and the two to four products half an ulp each: under 12 * 2^-24 more.  Below
# t = -87.3 the logistic, there under 1.2e-38, counts as 0.
def _rel(t):
    return (4 * t.abs().clamp(max=88) + 12) * 2.0 ** -24


def glu(rows, act, interleaved):
    """(h, bound of its float32 value)"""
    _, _, a, b, t, _, _ = _parts(rows, act, interleaved)
    h = a * torch.sigmoid(t) * b
    return h, _rel(t) * h.abs() + 2e-38 * (a * b).abs() + 2.0 ** -126


def glu_backward(g, rows, act, interleaved):
    """(gradient of the rows, bound of its float32 value)"""
    _, _, a, b, t, gate_in, up_in = _parts(rows, act, interleaved)
    g = g.double()
    s, rest = torch.sigmoid(t), torch.sigmoid(-t)
    gate, up = torch.where(gate_in, g * b * s * (1 + t * rest), 0.0), torch.where(up_in, g * a * s, 0.0)
    # 1 + t (1 - s): its terms may cancel, so their magnitudes count; 1 - s = e s has e's error twice
    e_gate = 2 * _rel(t) * (g * b * s).abs() * (1 + (t * rest).abs()) + 2e-38 * (g * b).abs() * (1 + t.abs()) + 2.0 ** -126
    e_up = _rel(t) * up.abs() + 2e-38 * (g * a).abs() + 2.0 ** -126
    return joined(gate, up, interleaved), joined(e_gate, e_up, interleaved)


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound, and half a step of got's type more for its rounding."""
    bound = bound + HALF_STEP[got.dtype] * 1.001 * (ref.abs() + bound)
    assert torch.isfinite(got).all(), what
    over = (got.double() - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: over the bound by {float(over.max()):.3e}"
