"""How far rows in 8 bits are off, as the calls state it, for blocks from the smallest subnormal to the largest
float32: half a step 2^(X - 7), which is 1/127 of a block's largest from 2^-127 on and stays 2^-134 below.  All
of it in float64, where these values and their differences are exact."""
import pytest
import torch

import rows_reference as ref

F32 = torch.float32


def _blocks():
    """Blocks whose largest is 1, 1.5, just under and at 127.5 / 64, and just under 2 times every power of two."""
    tops = torch.tensor([1.0, 1.5, 255 / 128 - 2.0 ** -22, 255 / 128, 2 - 2.0 ** -22], dtype=torch.float64)
    top = (tops[None] * torch.exp2(torch.arange(-149, 128, dtype=torch.float64))[:, None]).flatten()
    g = torch.Generator().manual_seed(1)
    part = torch.rand(len(top), 32, generator=g, dtype=torch.float64) * 2 - 1
    part[:, 0], part[:, 1], part[:, 2] = 1.0, -0.5, 2.0 ** -20
    return (part * top[:, None]).to(F32)


def _check(x, scales, back):
    x, back, byte = x.double(), back.double(), scales.double().reshape(-1)
    top, err = x.abs().amax(1), (back - x).abs().amax(1)
    assert torch.equal(byte == 0, top < 127.5 * 2.0 ** -133)
    saturates = top >= 2.0 ** 127 * 255 / 128
    assert (err <= torch.exp2(byte - 134))[~saturates].all()
    assert (back.abs().amax(1) == 127 * 2.0 ** 121)[saturates].all()
    assert (err <= top / 127)[top >= 2.0 ** -127].all()
    assert (err <= 2.0 ** -134)[top < 2.0 ** -127].all()
    assert (back == 0)[top <= 2.0 ** -134].all() and (top <= 2.0 ** -134).any()


def test_definition():
    x = _blocks()
    codes, scales = ref.rows8_of(x)
    _check(x, scales, ref.rows8_values(codes, scales))


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.bfloat16, F32])
def test_kernels(e4b, out):
    x = _blocks()
    codes, scales = e4b.e4b_checkpoint_rows(x.cuda())
    q, s = ref.rows8_of(x)
    assert torch.equal(codes.cpu(), q) and torch.equal(scales.cpu(), s)
    _check(x, scales.cpu(), e4b.e4b_restore_rows(codes, scales, dtype=out).cpu())
