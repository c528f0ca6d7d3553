"""The adapters' gradients with x kept in 8 bits: its values are bf16 values exactly, so every gradient has
the bits that the bf16 call gives for the restored rows."""
import numpy as np
import pytest
import torch

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def _normal(*shape, dtype=torch.bfloat16, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 64, 128])
@pytest.mark.parametrize("S,K,N,lengths,ids", [
    (1, 32, 8, [1], None),
    (100, 96, 64, [37, 0, 63], None),
    (900, 544, 72, [700, 129, 0, 71], [1, -1, 0, 1]),
    (513, 2880, 320, [513], None),
    (300, 256, 64, [100, 90, 80], [0, 0, 2])])
def test_same_bits_as_the_restored_rows(e4b, r, S, K, N, lengths, ids):
    n = len(lengths) if ids is None else max(ids) + 1
    codes, scales = e4b.e4b_checkpoint_rows(_normal(S, K, seed=1))
    x = e4b.e4b_restore_rows(codes, scales)
    g, z = _normal(S, N, seed=2), _normal(S, r, dtype=torch.float32, seed=3)
    a, b = _normal(n, r, K, seed=4, std=K ** -0.5), _normal(n, N, r, seed=5, std=r ** -0.5)
    scale = _normal(n, dtype=torch.float32, seed=6).abs()
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    ad = None if ids is None else torch.tensor(ids, dtype=torch.int32, device=DEV)
    base = _normal(S, K, dtype=torch.float32, seed=7)
    # in place: rows behind the last group are left as they were
    want = e4b.e4b_grouped_lora_backward(g, x, z, a, b, scale, off, ad, gx_base=(u := base.clone()), gx=u)
    got = e4b.e4b_grouped_lora_backward(g, codes, z, a, b, scale, off, ad, gx_base=(v := base.clone()), gx=v, x_scales=scales)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    only = e4b.e4b_grouped_lora_backward(g, codes, z, a, b, scale, off, ad, gx=False, gb=False, x_scales=scales)
    assert only[0] is None and only[2] is None and torch.equal(only[1], want[1])


def test_a_block_that_was_not_finite_is_nan_in_its_columns(e4b):
    S, K, N, r = 50, 96, 64, 16
    x = _normal(S, K, seed=1)
    x[20, 40] = float("inf")
    codes, scales = e4b.e4b_checkpoint_rows(x)
    args = (_normal(S, r, dtype=torch.float32, seed=3), _normal(1, r, K, seed=4), _normal(1, N, r, seed=5), None,
            torch.tensor([0, S], dtype=torch.int32, device=DEV))
    gx, ga, gb = e4b.e4b_grouped_lora_backward(_normal(S, N, seed=2), codes, *args, x_scales=scales)
    bad = torch.zeros(K, dtype=torch.bool, device=DEV)
    bad[32:64] = True
    assert torch.isnan(ga[:, :, bad]).all() and torch.isfinite(ga[:, :, ~bad]).all()
    assert torch.isfinite(gx).all() and torch.isfinite(gb).all()


def test_refusals(e4b):
    S, K, N, r = 8, 96, 64, 8
    codes, scales = e4b.e4b_checkpoint_rows(_normal(S, K, seed=1))
    g, z, a, b = _normal(S, N), _normal(S, r, dtype=torch.float32), _normal(1, r, K), _normal(1, N, r)
    off = torch.tensor([0, S], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        e4b.e4b_grouped_lora_backward(g, codes, z, a, b, None, off)                       # codes without scales
    with pytest.raises(ValueError):
        e4b.e4b_grouped_lora_backward(g, codes, z, a, b, None, off, x_scales=scales[:, :2].contiguous())
    with pytest.raises(ValueError):
        e4b.e4b_grouped_lora_backward(g, _normal(S, K), z, a, b, None, off, x_scales=scales)
    # x is not read without ga
    gx, ga, gb = e4b.e4b_grouped_lora_backward(g, None, z, a, b, None, off, ga=False, x_scales=scales)
    assert ga is None and torch.isfinite(gx).all() and torch.isfinite(gb).all()
