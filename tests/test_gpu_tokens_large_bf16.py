"""bf16 rows beyond what the memory-side cache keeps (270 MB, read past it): combine and its gradients."""
import pytest
import torch

from gpu_helpers import DEV
from test_gpu_tokens import BF16, F32, HALF_STEP, _assert_within, _combine64, _rows, _slots, _weights

pytestmark = pytest.mark.gpu

T, H, K, E = 9001, 3000, 5, 16


def test_combine(e4b):
    rows, slots, w = _rows(T * K, H, BF16, 60), _slots(T, K, E, 61), _weights(T, K, 62)
    assert rows.numel() * 2 > 256 << 20
    ref, mag = _combine64(rows, slots, K, w)
    bound = (K + 1) * 2.0 ** -24 * mag
    for dt in (BF16, F32):
        out = e4b.e4b_combine_tokens(rows, slots, K, w, dtype=dt)
        _assert_within(out, ref, bound + HALF_STEP[dt] * (ref.abs() + bound), "combine")


@pytest.mark.parametrize("g_t,d_t", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_combine_backward(e4b, g_t, d_t):
    g, rows, slots, w = _rows(T, H, g_t, 63), _rows(T * K, H, BF16, 60), _slots(T, K, E, 61), _weights(T, K, 62)
    g_rows, g_w = e4b.e4b_combine_tokens_backward(g, rows, slots, K, w, dtype=d_t)
    s = slots.long()
    gs = g.double()[s // K]
    ref = gs * w.double().reshape(-1)[s, None]
    _assert_within(g_rows, ref, (2.0 ** -24 + HALF_STEP[d_t] * 1.001) * ref.abs(), "g_rows")
    prod = gs * rows.double()
    _assert_within(g_w.reshape(-1)[s], prod.sum(1), (H + 1) * 2.0 ** -24 * prod.abs().sum(1), "g_w")
