"""The adapter calls on full-size layers, again and again: every pass gives the same bits, and the
first one the right values (a store that reads its registers too late shows in a pass of many)."""
import pytest
import torch

import test_gpu_lora as base
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r,dtype", [(8, base.F32), (16, base.F32), (32, base.F32), (64, base.F32), (128, base.F32),
                                     (8, base.BF16), (16, base.BF16), (32, base.BF16), (64, base.BF16), (128, base.BF16)])
def test_rows_of_a_layer(e4b, r, dtype):
    """8192 rows of 32 experts at [2880, 2880], an expert without an adapter among them."""
    lengths = [(131 * i) % 200 + 150 for i in range(31)]
    lengths.append(8192 - sum(lengths))
    p = base.Problem(K=2880, N=2880, r=r, lengths=lengths, ids=[i if i != 5 else -1 for i in range(32)], n=32)
    assert p.S == 8192 and lengths[-1] > 0
    y, g = base._normal(9, p.S, p.N, dtype=dtype), base._normal(10, p.S, p.N)
    z = base._normal(11, p.S, r, dtype=base.F32)
    args = (p.x, p.a, p.b, p.scale, p.offsets, p.ids)

    def step():
        return (e4b.e4b_grouped_lora(*args, y=y)[0], *e4b.e4b_grouped_lora_backward(g, p.x, z, *args[1:], gx_base=y))

    first = step()
    ref, bound, *_ = p.forward64(y)
    base._within(first[0], ref, bound, "out")
    for got, (ref, bound), what in zip(first[1:], p.backward64(g, z, y), ("gx", "ga", "gb")):
        base._within(got, ref, bound, what)
    for i in range(25):
        assert all(torch.equal(u, v) for u, v in zip(first, step())), i


@pytest.mark.parametrize("r", [8, 16, 32, 64])
def test_decoded_rows_of_a_layer(e4b, r):
    """512 rows of 128 experts, up to 16 rows each, in the one-launch form."""
    p = base.Problem(K=1024, N=14336, r=r, lengths=[(7 * i) % 9 for i in range(128)])
    y = base._normal(9, p.S, p.N, dtype=base.F32)

    def step():
        return e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, y=y)[0]

    first = step()
    ref, bound, *_ = p.forward64(y)
    base._within(first, ref, bound, "out")
    for i in range(25):
        assert torch.equal(first, step()), i
