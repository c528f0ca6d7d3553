"""Float32 rows to MXFP4 at every rounding boundary, bit for bit against the oracle."""
import numpy as np
import pytest
import torch

from gpu_helpers import DEV, host
from oracle import mxfp4 as omx

pytestmark = pytest.mark.gpu


def _check(e4b, x):
    blocks, scales = e4b.e4b_quantize_act_mxfp4(x)
    ob, os_ = omx.quantize_pack(host(x))
    assert np.array_equal(host(scales), os_) and np.array_equal(host(blocks), ob)


def test_halfway_values_and_their_neighbours(e4b):
    """Midpoints of neighbouring codes, a float32 step under and over them, in blocks from the smallest exponent to the largest."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.0, 7.9999995], dtype=torch.float32)
    near = torch.cat([mid, torch.nextafter(mid, mid * 0), torch.nextafter(mid, mid * 2)]).clamp(max=7.9999995)
    row = torch.zeros(32)
    row[:30] = near * torch.tensor([1.0, -1.0]).repeat(15)
    row[31] = 4.0
    exps = torch.arange(-149, 126, dtype=torch.float64)
    x = (row.double()[None] * torch.exp2(exps)[:, None]).float().to(DEV)
    _check(e4b, x)


def test_subnormal_rows(e4b):
    g = torch.Generator().manual_seed(1)
    bits = torch.randint(0, 1 << 23, (400, 64), generator=g, dtype=torch.int32) >> torch.randint(0, 23, (400, 1), generator=g, dtype=torch.int32)
    _check(e4b, bits.view(torch.float32).to(DEV))


def test_random_bits(e4b):
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-2 ** 31, 2 ** 31, (3000, 96), generator=g, dtype=torch.int64).to(torch.int32).view(torch.float32)
    _check(e4b, torch.where(torch.isfinite(x), x, torch.ones_like(x)).to(DEV))
