"""Adapter calls on a batch without rows, each set of outputs that a program may want."""
import itertools

import pytest
import torch

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gx,ga,gb", [w for w in itertools.product([None, False], repeat=3) if None in w])
def test_backward_without_rows(e4b, gx, ga, gb):
    a, b = torch.ones(3, 8, 64, dtype=torch.bfloat16, device=DEV), torch.ones(3, 48, 8, dtype=torch.bfloat16, device=DEV)
    x, g = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 48, dtype=torch.bfloat16, device=DEV)
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    got = e4b.e4b_grouped_lora_backward(g, x, torch.empty(0, 8, device=DEV), a, b, None, offsets, gx=gx, ga=ga, gb=gb)
    for wanted, t, shape in zip((gx, ga, gb), got, ((0, 64), a.shape, b.shape)):
        assert (t is None) if wanted is False else (t.shape == shape and bool((t == 0).all()))


def test_backward_that_wants_nothing_is_refused(e4b):
    a, b = torch.ones(1, 8, 64, dtype=torch.bfloat16, device=DEV), torch.ones(1, 48, 8, dtype=torch.bfloat16, device=DEV)
    for S in (0, 4):
        g = torch.ones(S, 48, dtype=torch.bfloat16, device=DEV)
        with pytest.raises(e4b.E4BError, match="status -1"):
            e4b.e4b_grouped_lora_backward(g, None, None, a, b, None, torch.tensor([0, S], dtype=torch.int32, device=DEV),
                                          gx=False, ga=False, gb=False)
