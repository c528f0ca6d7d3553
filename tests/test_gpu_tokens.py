"""Token permutation, combine and its gradients against float64, with bounds from the roundings:
a float32 sum of n products is off by at most n * 2^-24 of the sum of its terms' magnitudes, and a
bf16 result by half a step, 2^-8 of its value, more."""
import numpy as np
import pytest
import torch

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _slots(T, k, E, seed):
    """slot ids ordered by expert, then token, of random picks (an expert may have none)"""
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].reshape(-1)
    return torch.from_numpy(np.argsort(ids, kind="stable").astype(np.int32)).to(DEV)


def _rows(n, H, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(n, H, device=DEV, generator=g).to(dtype)


def _weights(T, k, seed):
    return torch.softmax(_rows(T, k, F32, seed), dim=1)


def _combine64(rows, slots, k, w):
    """(sum, sum of magnitudes) in float64; slots outside the range are dropped"""
    S, H = rows.shape
    s = slots.long()
    ok = (s >= 0) & (s < S)
    by_slot = torch.zeros(S, H, dtype=torch.float64, device=rows.device)
    by_slot[s[ok]] = rows.double()[ok]
    if w is not None:
        by_slot *= w.double().reshape(-1, 1)
    by_slot = by_slot.reshape(S // k, k, H)
    return by_slot.sum(1), by_slot.abs().sum(1)


def _assert_within(got, ref, bound, what):
    assert torch.isfinite(got).all(), what
    over = (got.double() - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: over the bound by {float(over.max()):.3e}"


# the last three have more than 4096 slots, the last one more than 65536 (other ways to find the rows)
SHAPES = [(1, 1, 1, 1), (1, 2048, 8, 128), (3, 7, 2, 4), (5, 64, 5, 5), (17, 1003, 3, 9), (300, 24, 4, 8),
          (512, 40, 8, 16), (513, 40, 8, 16), (1500, 520, 3, 7), (9001, 24, 8, 11)]


@pytest.mark.parametrize("T,H,k,E", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_permute_copies_the_rows(e4b, T, H, k, E, dtype):
    x, slots = _rows(T, H, dtype, 1), _slots(T, k, E, 2)
    rows = e4b.e4b_permute_tokens(x, slots, k)
    assert rows.dtype == dtype and torch.equal(rows, x[slots.long() // k])


@pytest.mark.parametrize("T,H,k,E", SHAPES)
@pytest.mark.parametrize("rows_t,out_t", [(F32, BF16), (BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(e4b, T, H, k, E, rows_t, out_t, weighted):
    rows, slots = _rows(T * k, H, rows_t, 3), _slots(T, k, E, 4)
    w = _weights(T, k, 5) if weighted else None
    out = e4b.e4b_combine_tokens(rows, slots, k, w, dtype=out_t)
    ref, mag = _combine64(rows, slots, k, w)
    bound = (k + 1) * 2.0 ** -24 * mag
    _assert_within(out, ref, bound + HALF_STEP[out_t] * (ref.abs() + bound), "combine")
    assert torch.equal(out, e4b.e4b_combine_tokens(rows, slots, k, w, dtype=out_t))  # same bits again


@pytest.mark.parametrize("T,H,k,E", SHAPES)
@pytest.mark.parametrize("g_t,rows_t,d_t", [(BF16, F32, BF16), (F32, BF16, F32), (BF16, BF16, F32), (F32, F32, BF16)])
def test_combine_backward(e4b, T, H, k, E, g_t, rows_t, d_t):
    g, rows, slots, w = _rows(T, H, g_t, 6), _rows(T * k, H, rows_t, 7), _slots(T, k, E, 8), _weights(T, k, 9)
    g_rows, g_w = e4b.e4b_combine_tokens_backward(g, rows, slots, k, w, dtype=d_t)
    s = slots.long()
    gs = g.double()[s // k]
    ref = gs * w.double().reshape(-1)[s, None]
    _assert_within(g_rows, ref, 2.0 ** -24 * ref.abs() + HALF_STEP[d_t] * 1.001 * ref.abs(), "g_rows")
    ref_w = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    mag_w = torch.zeros_like(ref_w)
    ref_w[s], mag_w[s] = (gs * rows.double()).sum(1), (gs * rows.double()).abs().sum(1)
    _assert_within(g_w.reshape(-1), ref_w, (H + 1) * 2.0 ** -24 * mag_w, "g_w")
    frozen, none = e4b.e4b_combine_tokens_backward(g, None, slots, k, w, dtype=d_t)
    assert none is None and torch.equal(frozen, g_rows)


def test_combine_gradients_against_differences(e4b):
    """The combine is linear in the rows and in the weights: <g, change of out> equals the
    gradients' products with the changes, up to the roundings."""
    T, H, k, E = 37, 72, 3, 6
    rows, slots, w, g = _rows(T * k, H, F32, 10), _slots(T, k, E, 11), _weights(T, k, 12), _rows(T, H, F32, 13)
    dr, dw = _rows(T * k, H, F32, 14), _rows(T, k, F32, 15)
    g_rows, g_w = e4b.e4b_combine_tokens_backward(g, rows, slots, k, w, dtype=F32)
    f = lambda r, ww: e4b.e4b_combine_tokens(r, slots, k, ww, dtype=F32).double()
    for change, grad, step in ((f(rows + dr, w) - f(rows, w), g_rows, dr), (f(rows, w + dw) - f(rows, w), g_w, dw)):
        left, right = float((g.double() * change).sum()), float((grad.double() * step.double()).sum())
        # each out value is a sum of k <= 3 terms of magnitude <= ~30: a few hundred float32
        # roundings of 30 * 2^-24, weighted by |g| <= ~5 over T * H values
        assert abs(left - right) <= T * H * 5 * 30 * 8 * 2.0 ** -24


@pytest.mark.parametrize("T", [40, 2000, 20000])
def test_slots_without_a_row_and_named_twice(e4b, T):
    """A dropped row (slot -1 or past the end) contributes nothing and is left alone; of two rows
    that name one slot the higher counts."""
    H, k, E = 48, 4, 8
    slots = _slots(T, k, E, 16)
    slots[3], slots[10], slots[T] = -1, T * k, 2 ** 31 - 1
    slots[7] = slots[20]                                 # row 20 counts
    x, rows, w, g = _rows(T, H, BF16, 17), _rows(T * k, H, F32, 18), _weights(T, k, 19), _rows(T, H, BF16, 20)
    s = slots.long()
    named = (s >= 0) & (s < T * k)
    got = e4b.e4b_permute_tokens(x, slots, k)
    assert torch.equal(got, torch.where(named[:, None], x[torch.where(named, s, 0) // k], torch.zeros_like(got)))
    used = s.clone()
    used[7] = -1
    out = e4b.e4b_combine_tokens(rows, slots, k, w, dtype=F32)
    ref, mag = _combine64(rows, used, k, w)
    _assert_within(out, ref, (k + 2) * 2.0 ** -24 * mag, "combine")
    g_rows = torch.full((T * k, H), 7.0, device=DEV)
    g_w = torch.full((T, k), 7.0, device=DEV)
    e4b.e4b_combine_tokens_backward(g, rows, slots, k, w, g_rows=g_rows, g_w=g_w)
    for p in (3, 10, T, 7):
        assert (g_rows[p] == 7.0).all()
    missing = torch.ones(T * k, dtype=torch.bool, device=DEV)
    missing[used[(used >= 0) & (used < T * k)]] = False
    assert (g_w.reshape(-1)[missing] == 0).all() and int(missing.sum()) == 4


@pytest.mark.parametrize("T,H,k", [(4100, 2051, 8), (70000, 520, 2), (600000, 31, 4)])
def test_permute_in_token_order(e4b, T, H, k):
    """From 128 MB of rows the rows are written token by token; dropped rows and a slot named twice as above."""
    x, slots = _rows(T, H, BF16, 50), _slots(T, k, 16, 51)
    assert e4b.e4b_permute_workspace_bytes(T, H, k) > 0
    out = torch.full((T * k, H), 7.0, dtype=BF16, device=DEV)
    assert torch.equal(e4b.e4b_permute_tokens(x, slots, k, out=out), x[slots.long() // k])
    slots[3], slots[T], slots[T * k - 1], slots[70] = -1, T * k, 2 ** 31 - 1, slots[9000]
    s = slots.long()
    named = (s >= 0) & (s < T * k)
    got = e4b.e4b_permute_tokens(x, slots, k, out=out.fill_(7.0))
    assert torch.equal(got, torch.where(named[:, None], x[torch.where(named, s, 0) // k], torch.zeros_like(got)))


def test_more_rows_than_the_cache_keeps(e4b):
    """Rows of 275 MB (read past the caches): combine and its gradients."""
    T, H, k, E = 16500, 521, 8, 16
    rows, slots, w, g = _rows(T * k, H, F32, 60), _slots(T, k, E, 61), _weights(T, k, 62), _rows(T, H, BF16, 63)
    out = e4b.e4b_combine_tokens(rows, slots, k, w, dtype=F32)
    ref, mag = _combine64(rows, slots, k, w)
    _assert_within(out, ref, (k + 2) * 2.0 ** -24 * mag, "combine")
    del ref, mag, out
    g_rows, g_w = e4b.e4b_combine_tokens_backward(g, rows, slots, k, w)
    s = slots.long()
    gs = g.double()[s // k]
    ref = gs * w.double().reshape(-1)[s, None]
    _assert_within(g_rows, ref, (2.0 ** -24 + HALF_STEP[BF16] * 1.001) * ref.abs(), "g_rows")
    prod = gs * rows.double()
    assert ((g_w.double().reshape(-1)[s] - prod.sum(1)).abs() <= (H + 1) * 2.0 ** -24 * prod.abs().sum(1)).all()


def test_infinities_stay_in_their_rows(e4b):
    T, H, k, E = 20, 16, 2, 4
    slots, w = _slots(T, k, E, 21), _weights(T, k, 22)
    rows = _rows(T * k, H, F32, 23)
    rows[5], rows[9, 3] = float("inf"), float("nan")
    for dt in (BF16, F32):
        out = e4b.e4b_combine_tokens(rows, slots, k, w, dtype=dt)
        bad = torch.zeros(T, H, dtype=torch.bool, device=DEV)
        bad[int(slots[5]) // k] = True
        bad[int(slots[9]) // k, 3] = True
        assert torch.equal(torch.isfinite(out), ~bad) and torch.isnan(out[int(slots[9]) // k, 3])


@pytest.mark.parametrize("T", [16, 1100])
def test_on_another_stream_and_captured(e4b, T):
    """The calls on a side stream, and a captured sequence replayed with eager work in between."""
    H, k, E = 256, 4, 8
    x, slots, w = _rows(T, H, BF16, 24), _slots(T, k, E, 25), _weights(T, k, 26)

    def step(**kw):
        rows = e4b.e4b_permute_tokens(x, slots, k, **kw)
        out = e4b.e4b_combine_tokens(rows, slots, k, w, **kw)
        return (rows, out, *e4b.e4b_combine_tokens_backward(out, rows, slots, k, w, **kw))

    eager = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(3):
        x.copy_(_rows(T, H, BF16, 30 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, step())), i


def test_empty_batch(e4b):
    slots, w = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV)
    x = torch.empty(0, 8, dtype=BF16, device=DEV)
    rows = e4b.e4b_permute_tokens(x, slots, 2)
    assert rows.shape == (0, 8) and e4b.e4b_combine_tokens(rows, slots, 2, w).shape == (0, 8)
    g_rows, g_w = e4b.e4b_combine_tokens_backward(x, rows, slots, 2, w)
    assert g_rows.shape == (0, 8) and g_w.shape == (0, 2)


def test_binding_refuses(e4b):
    T, H, k = 6, 16, 2
    x, slots, w = _rows(T, H, BF16, 1), _slots(T, k, 4, 2), _weights(T, k, 3)
    rows = _rows(T * k, H, F32, 4)
    for f in (lambda: e4b.e4b_permute_tokens(_rows(H, T, BF16, 1).t(), slots, k),  # strided
              lambda: e4b.e4b_permute_tokens(x.half(), slots, k),
              lambda: e4b.e4b_permute_tokens(x, slots.long(), k),
              lambda: e4b.e4b_permute_tokens(x, slots, 3),
              lambda: e4b.e4b_permute_tokens(x, slots, k, out=rows),
              lambda: e4b.e4b_combine_tokens(rows, slots, 5, w),
              lambda: e4b.e4b_combine_tokens(rows, slots, k, w.to(BF16)),
              lambda: e4b.e4b_combine_tokens(rows, slots, k, w[:3]),
              lambda: e4b.e4b_combine_tokens(rows, slots, k, w, dtype=torch.float16),
              lambda: e4b.e4b_combine_tokens_backward(x, rows[:4], slots, k, w),
              lambda: e4b.e4b_combine_tokens_backward(x, None, slots, k, w, g_w=w)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        e4b.e4b_combine_tokens_backward(x, rows, slots, k, None)
    for f in (lambda: e4b.e4b_permute_tokens(_rows(1, H, BF16, 1), torch.zeros(65, dtype=torch.int32, device=DEV), 65),
              lambda: e4b.e4b_combine_tokens(torch.empty(T * k * H + 1, device=DEV)[1:].view(T * k, H), slots, k, w)):
        with pytest.raises(e4b.E4BError):
            f()


def test_routed_layer_order(e4b):
    """permute and combine with the slots of e4b_route_permute: identity experts give each token
    back, weighted by weights that sum to one."""
    T, H, k, E = 77, 128, 2, 8
    x = _rows(T, H, BF16, 40)
    _, w, _, slots = e4b.e4b_route_permute(_rows(T, E, F32, 41), k)
    out = e4b.e4b_combine_tokens(e4b.e4b_permute_tokens(x, slots, k), slots, k, w, dtype=F32)
    bound = (k + 3) * 2.0 ** -24 * 2 * x.double().abs()
    _assert_within(out, x.double(), bound, "identity experts")
