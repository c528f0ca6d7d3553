"""Grouped low-rank adapters and their gradients against float64.  Bounds: a product of two bf16
values is exact in float32; a float32 sum of n terms is off by at most n * 2^-23 of the sum of
their magnitudes (2^-23: whichever way the matrix unit rounds an addition); a result of type t by
half a step of t, `torch.finfo(t).eps / 2`, of its value more.  z and u enter their second product
as three parts that hold all 24 bits, so nothing else is rounded."""
import numpy as np
import pytest
import torch

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -23


def _normal(seed, *shape, dtype=BF16, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


class Problem:
    """lengths: rows of each group; before / after: rows outside every group."""

    def __init__(self, K, N, r, lengths, ids=None, n=None, before=0, after=0, seed=0):
        offsets = before + np.concatenate([[0], np.cumsum(lengths)])
        self.S, self.K, self.N, self.r = int(offsets[-1]) + after, K, N, r
        self.offsets_np = offsets
        self.ids_np = list(range(len(lengths))) if ids is None else list(ids)
        self.n = n if n is not None else max(len(lengths) if ids is None else max(ids) + 1, 1)
        self.offsets = torch.from_numpy(offsets.astype(np.int32)).to(DEV)
        self.ids = None if ids is None else torch.tensor(ids, dtype=torch.int32, device=DEV)
        self.x = _normal(seed + 1, self.S, K)
        self.a = _normal(seed + 2, self.n, r, K, std=K ** -0.5)
        self.b = _normal(seed + 3, self.n, N, r, std=r ** -0.5)
        self.scale = torch.rand(self.n, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)) + 0.5
        self.seed = seed

    def groups(self):
        """(rows, adapter) of the groups with rows and an adapter"""
        for lo, hi, i in zip(self.offsets_np[:-1], self.offsets_np[1:], self.ids_np):
            if hi > lo and 0 <= i < self.n:
                yield slice(int(lo), int(hi)), i

    def forward64(self, y):
        """out, its bound before the last rounding, z, z's bound; float64"""
        S, x, a, b, s = self.S, self.x.double(), self.a.double(), self.b.double(), self.scale.double()
        out = torch.zeros(S, self.N, dtype=torch.float64, device=DEV) if y is None else y.double()
        z = torch.zeros(S, self.r, dtype=torch.float64, device=DEV)
        zb, ob = torch.zeros_like(z), torch.zeros_like(out)
        for rows, i in self.groups():
            z[rows] = x[rows] @ a[i].T
            zb[rows] = (self.K + 1) * E * (x[rows].abs() @ a[i].abs().T)
            mag = s[i] * (z[rows].abs() @ b[i].abs().T)
            ob[rows] = s[i] * (zb[rows] @ b[i].abs().T) + (3 * self.r + 4) * E * mag
            out[rows] += s[i] * (z[rows] @ b[i].T)
        return out, ob * 1.01, z, zb

    def backward64(self, g, z, base):
        x, a, b, s = self.x.double(), self.a.double(), self.b.double(), self.scale.double()
        g, z = g.double(), z.double()
        gx = torch.zeros(self.S, self.K, dtype=torch.float64, device=DEV) if base is None else base.double()
        gxb, ga, gb = torch.zeros_like(gx), torch.zeros_like(a), torch.zeros_like(b)
        gab, gbb, rows_of = torch.zeros_like(a), torch.zeros_like(b), [0] * self.n
        for rows, i in self.groups():
            rows_of[i] += rows.stop - rows.start
        for rows, i in self.groups():
            u = s[i] * (g[rows] @ b[i])
            ub = (self.N + 3) * E * s[i] * (g[rows].abs() @ b[i].abs())
            gx[rows] += u @ a[i]
            gxb[rows] = ub @ a[i].abs() + (3 * self.r + 4) * E * (u.abs() @ a[i].abs())
            ga[i] += u.T @ x[rows]
            gab[i] += ub.T @ x[rows].abs() + (rows_of[i] + 4) * E * (u.abs().T @ x[rows].abs())
            gb[i] += s[i] * (g[rows].T @ z[rows])
            gbb[i] += (rows_of[i] + 4) * E * s[i] * (g[rows].abs().T @ z[rows].abs())
        return (gx, gxb * 1.01), (ga, gab * 1.01), (gb, gbb * 1.01)


def _within(got, ref, bound, what):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = bound + torch.finfo(got.dtype).eps / 2 * (ref.abs() + bound)
    over = (got.double() - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: over the bound by {float(over.max()):.3e} at {int(over.argmax())}"


CASES = {
    "one_row": dict(K=8, N=8, r=8, lengths=[1]),
    "one_token_wide": dict(K=4096, N=1032, r=16, lengths=[1]),
    "tile_edges": dict(K=64, N=72, r=16, lengths=[0, 1, 16, 17, 63, 64, 65, 0, 129]),
    "odd_columns": dict(K=1032, N=40, r=24, lengths=[70, 3, 90]),
    "rank_8": dict(K=136, N=520, r=8, lengths=[33, 200]),
    "rank_32": dict(K=520, N=136, r=32, lengths=[100, 0, 41]),
    "rank_64": dict(K=256, N=264, r=64, lengths=[5, 150]),
    "rank_72": dict(K=96, N=64, r=72, lengths=[31, 33, 97]),
    "rank_128": dict(K=320, N=192, r=128, lengths=[64, 40, 200]),
    "decode_requests": dict(K=1024, N=256, r=16, lengths=[1] * 70, ids=[(7 * i) % 20 if i % 9 else -1 for i in range(70)], n=20),
    "many_groups": dict(K=48, N=56, r=40, lengths=[(3 * i) % 7 for i in range(200)]),
    "shared_adapters": dict(K=128, N=80, r=16, lengths=[40, 0, 100, 7, 200, 65], ids=[1, 0, 3, 1, -1, 3], n=5),
    "rows_outside": dict(K=72, N=48, r=16, lengths=[20, 30], before=7, after=19),
    "fewer_adapters_than_groups": dict(K=72, N=48, r=16, lengths=[20, 30, 9], n=2),
    "more_adapters_than_groups": dict(K=72, N=48, r=8, lengths=[20, 80], n=4),
    "one_group": dict(K=2048, N=512, r=16, lengths=[700]),
}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", CASES)
def test_forward(e4b, name, dtype):
    p = Problem(**CASES[name])
    y = _normal(9, p.S, p.N, dtype=dtype)
    ref, bound, zref, zbound = p.forward64(y)
    out, z = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, y=y, z=True,
                                  out=torch.full_like(y, 7.0))
    lo, hi = int(p.offsets_np[0]), int(p.offsets_np[-1])
    _within(out[lo:hi], ref[lo:hi], bound[lo:hi], "out")
    _within(z[lo:hi], zref[lo:hi], zbound[lo:hi], "z")
    assert (out[:lo] == 7.0).all() and (out[hi:] == 7.0).all()  # rows of no group stay as they were
    # in place, and the same bits without z
    again = y.clone()
    got, none = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, y=again, out=again)
    assert none is None and got is again and torch.equal(again[lo:hi], out[lo:hi])
    assert torch.equal(again[:lo], y[:lo]) and torch.equal(again[hi:], y[hi:])
    # without a projection
    delta, _ = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, dtype=dtype)
    ref, bound, *_ = p.forward64(None)
    assert delta.dtype == dtype
    _within(delta[lo:hi], ref[lo:hi], bound[lo:hi], "delta")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", CASES)
def test_backward(e4b, name, dtype):
    p = Problem(**CASES[name])
    g, z, base = _normal(10, p.S, p.N), _normal(11, p.S, p.r, dtype=F32), _normal(12, p.S, p.K, dtype=dtype)
    refs = p.backward64(g, z, base)
    args = (g, p.x, z, p.a, p.b, p.scale, p.offsets, p.ids)
    lo, hi = int(p.offsets_np[0]), int(p.offsets_np[-1])
    gx, ga, gb = e4b.e4b_grouped_lora_backward(*args, gx_base=base, gx=torch.full_like(base, 7.0),
                                               ga=torch.full_like(p.a, 7.0, dtype=F32))
    _within(gx[lo:hi], refs[0][0][lo:hi], refs[0][1][lo:hi], "gx")
    _within(ga, *refs[1], "ga")
    _within(gb, *refs[2], "gb")
    assert (gx[:lo] == 7.0).all() and (gx[hi:] == 7.0).all()
    again = e4b.e4b_grouped_lora_backward(*args, gx_base=base)
    assert torch.equal(again[0][lo:hi], gx[lo:hi]) and torch.equal(again[1], ga) and torch.equal(again[2], gb)
    place = base.clone()
    e4b.e4b_grouped_lora_backward(*args, gx_base=place, gx=place, ga=False, gb=False)
    assert torch.equal(place[lo:hi], gx[lo:hi])
    # each output alone
    assert torch.equal(e4b.e4b_grouped_lora_backward(g, None, z, *args[3:], gx=False, ga=False)[2], gb)
    alone = e4b.e4b_grouped_lora_backward(g, p.x, None, *args[3:], gx=False, gb=False)
    _within(alone[1], *refs[1], "ga alone")
    assert alone[0] is None and alone[2] is None
    gx0 = e4b.e4b_grouped_lora_backward(*args, ga=False, gb=False, dtype=dtype)[0]
    (ref, bound), *_ = p.backward64(g, z, None)
    _within(gx0[lo:hi], ref[lo:hi], bound[lo:hi], "gx without a base")


def test_no_scale_is_scale_one(e4b):
    p = Problem(**CASES["shared_adapters"])
    one = torch.ones(p.n, device=DEV)
    g, z = _normal(10, p.S, p.N), _normal(11, p.S, p.r, dtype=F32)
    lo, hi = int(p.offsets_np[0]), int(p.offsets_np[-1])
    f = lambda s: e4b.e4b_grouped_lora(p.x, p.a, p.b, s, p.offsets, p.ids)[0][lo:hi]
    assert torch.equal(f(None), f(one))
    h = lambda s: e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, s, p.offsets, p.ids)
    assert all(torch.equal(u, v) for u, v in zip(h(None), h(one)))


def test_gradients_against_differences(e4b):
    """out is linear in x, in a and in b each: the change of <g, out> under a finite change of one
    of them is the product of its gradient with the change, up to the roundings above."""
    p = Problem(K=64, N=48, r=8, lengths=[20, 0, 37, 5], ids=[1, 0, 1, -1], n=2, seed=5)
    g = _normal(10, p.S, p.N)
    rows = slice(0, p.S)

    def out(x, a, b):
        return e4b.e4b_grouped_lora(x, a, b, p.scale, p.offsets, p.ids)[0].double()

    z = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, z=True)[1]
    gx, ga, gb = e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, p.scale, p.offsets, p.ids)
    first = out(p.x, p.a, p.b)
    bound = p.forward64(None)[1]
    for name, grad, t in (("x", gx, p.x), ("a", ga, p.a), ("b", gb, p.b)):
        moved = (t.float() + _normal(20, *t.shape, dtype=F32, std=0.5)).to(BF16)
        step = moved.double() - t.double()
        new = {"x": p.x, "a": p.a, "b": p.b, name: moved}
        change = float((g.double() * (out(**new) - first)).sum())
        # each out value of either call is within `bound` (times 4 for the larger operands)
        slack = 10 * float((g.double().abs() * bound)[rows].sum()) + 1e-6
        assert abs(change - float((grad.double() * step).sum())) <= slack, name


@pytest.mark.parametrize("where", ["x", "y", "g"])
def test_nan_and_infinity_stay_in_their_row(e4b, where):
    """A NaN or infinity in a row reaches that row alone, and the gradients of its adapter alone."""
    p = Problem(K=96, N=64, r=16, lengths=[21, 50, 3], seed=3)
    y, g, z = _normal(9, p.S, p.N, dtype=F32), _normal(10, p.S, p.N), _normal(11, p.S, p.r, dtype=F32)
    row, bad = 30, torch.zeros(p.S, dtype=torch.bool, device=DEV)
    bad[row] = True
    {"x": p.x, "y": y, "g": g}[where][row, 5] = float("nan") if where != "y" else float("inf")
    out, _ = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, y=y)
    gx, ga, gb = e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, p.scale, p.offsets)
    if where == "y":
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[row, 5] = True
        assert torch.equal(torch.isfinite(out), ~hit)
        return
    if where == "x":
        assert torch.equal(torch.isfinite(out).all(1), ~bad) and torch.isfinite(gx).all() and torch.isfinite(gb).all()
        assert torch.isfinite(ga[0]).all() and torch.isfinite(ga[2]).all()
        assert torch.equal(torch.isfinite(ga[1]).all(0), torch.arange(p.K, device=DEV) != 5)
    else:
        assert torch.equal(torch.isfinite(gx).all(1), ~bad)
        assert torch.isfinite(ga[[0, 2]]).all() and torch.isfinite(gb[[0, 2]]).all()
        assert torch.equal(torch.isfinite(gb[1]).all(1), torch.arange(p.N, device=DEV) != 5)


@pytest.mark.parametrize("r", [16, 64, 104])
def test_what_is_outside_does_not_reach_the_results(e4b, r):
    """NaN in rows of no group, in rows of groups without an adapter and in the workspace."""
    p = Problem(K=160, N=144, r=r, lengths=[21, 50, 3, 70, 130], ids=[1, -1, 0, 1, 5], n=3, before=5, after=40)
    y, g, z = _normal(9, p.S, p.N, dtype=F32), _normal(10, p.S, p.N), _normal(11, p.S, p.r, dtype=F32)
    inside = torch.zeros(p.S, dtype=torch.bool, device=DEV)
    for rows, _ in p.groups():
        inside[rows] = True

    def step(x, g, z, byte):
        sizes = (p.S, p.K, p.N, p.r, 5, 3)
        ws = [torch.full((n,), byte, dtype=torch.uint8, device=DEV)
              for n in (max(16, e4b.e4b_lora_workspace_bytes(*sizes)), e4b.e4b_lora_backward_workspace_bytes(*sizes, True))]
        out = e4b.e4b_grouped_lora(x, p.a, p.b, p.scale, p.offsets, p.ids, y=y, ws=ws[0])[0]
        gx, ga, gb = e4b.e4b_grouped_lora_backward(g, x, z, p.a, p.b, p.scale, p.offsets, p.ids, ws=ws[1])
        return out[inside], gx[inside], ga, gb

    clean = step(p.x, g, z, 0)
    soiled = []
    for t in (p.x, g, z):
        t = t.clone()
        t[~inside] = float("nan")
        soiled.append(t)
    assert all(torch.isfinite(t).all() for t in clean)
    assert all(torch.equal(u, v) for u, v in zip(clean, step(*soiled, 0xFF)))


def test_binding_refuses(e4b):
    p = Problem(K=64, N=48, r=8, lengths=[20, 30])
    y, g, z = _normal(9, p.S, p.N), _normal(10, p.S, p.N), _normal(11, p.S, p.r, dtype=F32)
    head, tail = (p.x, p.a, p.b), (p.scale, p.offsets)
    wide = torch.empty(p.S, 2 * p.K, dtype=BF16, device=DEV)
    for kind, args, kw in (
            (ValueError, (wide[:, :64], p.a, p.b, *tail), {}),                      # strided
            (ValueError, (p.x.float(), p.a, p.b, *tail), {}),
            (ValueError, (p.x, p.a[:, :, :56].contiguous(), p.b, *tail), {}),
            (ValueError, (p.x, p.a, p.b[:1].contiguous(), *tail), {}),
            (ValueError, (*head, p.scale[:1].contiguous(), p.offsets), {}),
            (ValueError, (*head, p.scale, p.offsets.long()), {}),
            (ValueError, (*head, p.scale, p.offsets[:1]), {}),
            (ValueError, (*head, *tail), {"y": y, "dtype": F32, "out": y.float()}),
            (ValueError, (*head, *tail), {"dtype": torch.float16}),
            (ValueError, (*head, *tail), {"z": torch.empty(p.S, 16, device=DEV)}),
            (e4b.E4BError, (*head, *tail), {"out": torch.empty(p.S * p.N + 1, device=DEV)[1:].view(p.S, p.N)}),
            (e4b.E4BError, (p.x, torch.cat([p.a, p.a[:, :4]], 1), torch.cat([p.b, p.b[:, :, :4]], 2), *tail), {})):
        with pytest.raises(kind):
            e4b.e4b_grouped_lora(*args, **kw)
    for kind, args, kw in (
            (ValueError, (g.t(), p.x, z, p.a, p.b, *tail), {}),
            (TypeError, (g, None, z, p.a, p.b, *tail), {}),
            (TypeError, (g, p.x, None, p.a, p.b, *tail), {}),
            (ValueError, (g, p.x, z, p.a, p.b, *tail), {"gx": False, "gx_base": p.x}),
            (ValueError, (g, p.x, z, p.a, p.b, *tail), {"gx": p.x.float(), "gx_base": p.x}),
            (ValueError, (g, p.x, z, p.a, p.b, *tail), {"ga": p.a}),
            (e4b.E4BError, (g, p.x, z, p.a, p.b, *tail), {"gx": False, "ga": False, "gb": False}),
            (e4b.E4BError, (g, p.x, z, p.a, p.b, *tail), {"ws": torch.empty(16, dtype=torch.uint8, device=DEV)})):
        with pytest.raises(kind):
            e4b.e4b_grouped_lora_backward(*args, **kw)


def test_empty_batch_and_empty_groups(e4b):
    p = Problem(K=64, N=48, r=8, lengths=[0, 0, 0])
    assert p.S == 0
    out, z = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, z=True)
    assert out.shape == (0, 48) and z.shape == (0, 8)
    g = torch.empty(0, 48, dtype=BF16, device=DEV)
    gx, ga, gb = e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, p.scale, p.offsets, ga=_normal(1, 3, 8, 64, dtype=F32),
                                               gb=_normal(1, 3, 48, 8, dtype=F32))
    assert gx.shape == (0, 64) and (ga == 0).all() and (gb == 0).all()
    # rows, but all of them outside the groups
    q = Problem(K=64, N=48, r=8, lengths=[0, 0], after=30)
    g = _normal(2, 30, 48)
    gx, ga, gb = e4b.e4b_grouped_lora_backward(g, q.x, torch.zeros(30, 8, device=DEV), q.a, q.b, q.scale, q.offsets,
                                               gx=torch.full((30, 64), 7.0, device=DEV))
    assert (gx == 7.0).all() and (ga == 0).all() and (gb == 0).all()


def test_offsets_are_clamped_to_the_rows(e4b):
    """Offsets past the last row name the rows there are."""
    p = Problem(K=64, N=48, r=8, lengths=[40, 60])
    over = torch.tensor([-5, 40, 400], dtype=torch.int32, device=DEV)
    g, z = _normal(2, p.S, p.N), _normal(3, p.S, p.r, dtype=F32)
    for f in (lambda o: e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, o)[:1],
              lambda o: e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, p.scale, o)):
        assert all(torch.equal(u, v) for u, v in zip(f(over), f(p.offsets)))


def test_other_stream_and_captured(e4b):
    p = Problem(K=1024, N=264, r=16, lengths=[100, 0, 30, 300])
    y, g = _normal(9, p.S, p.N, dtype=F32), _normal(10, p.S, p.N)

    def step(**kw):
        out, z = e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, y=y, z=True, **kw)
        return (out, z, *e4b.e4b_grouped_lora_backward(g, p.x, z, p.a, p.b, p.scale, p.offsets, **kw))

    eager = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = step(stream=side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(3):
        p.x.copy_(_normal(30 + i, p.S, p.K))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(captured, step())), i


def test_wide_rows_pass_32_bit_offsets(e4b):
    """S * N beyond 2^31 elements: the last rows of a tall out."""
    S, K, N, r = 70001, 64, 32768, 8
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    x, a, b = _normal(1, S, K), _normal(2, 1, r, K, std=K ** -0.5), _normal(3, 1, N, r, std=r ** -0.5)
    offsets = torch.tensor([0, S], dtype=torch.int32, device=DEV)
    out, _ = e4b.e4b_grouped_lora(x, a, b, None, offsets, dtype=BF16)
    tail = slice(S - 40, S)
    z = x[tail].double() @ a[0].double().T
    ref = z @ b[0].double().T
    bound = (K + 1) * E * (x[tail].double().abs() @ a[0].double().abs().T) @ b[0].double().abs().T
    bound += (3 * r + 4) * E * (z.abs() @ b[0].double().abs().T)
    _within(out[tail], ref, bound * 1.01, "tail")
    g = out  # bf16 [S, N]
    gb = e4b.e4b_grouped_lora_backward(g, None, torch.ones(S, r, device=DEV), a, b, None, offsets, gx=False, ga=False)[2]
    cols = slice(N - 16, N)
    ref = g[:, cols].double().sum(0)
    bound = (S + 4) * E * g[:, cols].double().abs().sum(0)
    _within(gb[0, cols, 0], ref, bound, "gb")
