"""Rows of a group without an adapter are copies, bit for bit: the sign of a zero included."""
import pytest
import torch

import test_gpu_lora as base
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", [base.F32, base.BF16])
@pytest.mark.parametrize("r,lengths", [(16, [1, 3, 2]), (16, [70, 33, 129]), (72, [4, 2, 9]), (72, [70, 33, 129])])
def test_rows_without_an_adapter_are_copies(e4b, r, lengths, dtype):
    p = base.Problem(K=72, N=136, r=r, lengths=lengths, ids=[0, -1, 5], n=2)
    bare = slice(lengths[0], p.S)
    y, gx0 = base._normal(9, p.S, p.N, dtype=dtype), base._normal(12, p.S, p.K, dtype=dtype)
    for t in (y, gx0):
        t[:, ::3], t[:, 1::7] = -0.0, 0.0
        t[-1, 2:5] = torch.tensor([float("inf"), -float("inf"), torch.finfo(dtype).tiny], device=DEV).to(dtype)
    g, z = base._normal(10, p.S, p.N), base._normal(11, p.S, r, dtype=base.F32)
    out, _ = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, y=y)
    gx, _, _ = e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, p.scale, p.offsets, p.ids, gx_base=gx0)
    assert torch.equal(_bits(out[bare]), _bits(y[bare])) and torch.equal(_bits(gx[bare]), _bits(gx0[bare]))
    # without a base they are zeros
    out, _ = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, dtype=dtype)
    assert (_bits(out[bare]) == 0).all()
