"""What is no tensor is refused as such, for every tensor the adapter calls take."""
import pytest
import torch

import test_gpu_lora as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [[1.0], 3, "y"])
def test_arguments_that_are_no_tensors(e4b, bad):
    p = base.Problem(K=64, N=48, r=8, lengths=[5])
    g, z = base._normal(10, p.S, p.N), base._normal(11, p.S, p.r, dtype=base.F32)
    head, back = [p.x, p.a, p.b, p.scale, p.offsets], [g, p.x, z, p.a, p.b, p.scale, p.offsets]
    for f, args, names in ((e4b.e4b_grouped_lora, head, ("group_adapter", "y", "out", "z", "ws")),
                           (e4b.e4b_grouped_lora_backward, back, ("group_adapter", "gx_base", "gx", "ga", "gb", "ws"))):
        for i in range(len(args)):
            with pytest.raises(TypeError):
                f(*args[:i], bad, *args[i + 1:])
        for name in names:
            with pytest.raises(TypeError):
                f(*args, **{name: bad})
