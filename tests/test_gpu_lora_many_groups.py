"""As many groups as the adapter calls take, nearly all of them empty."""
import numpy as np
import pytest
import torch

import test_gpu_lora as base
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r,K", [(16, 136), (72, 264)])
def test_many_groups(e4b, r, K):
    G, n, N = 65536, 5, 72
    rng = np.random.default_rng(r)
    lengths = np.zeros(G, dtype=np.int64)
    for g in (0, 63, 64, 4095, 4096, 40000, G - 1):
        lengths[g] = rng.integers(1, 40)
    ids = rng.integers(-1, n, G)
    ids[[0, G - 1]] = 1, 4
    p = base.Problem(K=K, N=N, r=r, lengths=lengths, ids=ids.tolist(), n=n)
    y, g, z = base._normal(9, p.S, N, dtype=base.F32), base._normal(10, p.S, N), base._normal(11, p.S, r, dtype=base.F32)
    ref, bound, zref, zbound = p.forward64(y)
    out, zout = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, y=y, z=True)
    base._within(out, ref, bound, "out")
    base._within(zout, zref, zbound, "z")
    gx0 = base._normal(12, p.S, K, dtype=base.F32)
    for got, (want, off), what in zip(e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, p.scale, p.offsets, p.ids, gx_base=gx0),
                                      p.backward64(g, z, gx0), ("gx", "ga", "gb")):
        base._within(got, want, off, what)
