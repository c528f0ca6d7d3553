"""The adapter calls through each form that the sizes choose between: decoded tokens in one launch
at every rank it takes, decoded tokens in two launches (a wide A, or ranks over 64), columns cut into
sixteen pieces, and groups of very unequal lengths.  Bounds as in test_gpu_lora."""
import pytest
import torch

import test_gpu_lora as base
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

FORMS = {
    # one launch (at most 16 rows a group on average, rank up to 64, r K up to 2^17)
    "one_launch_8": dict(K=1032, N=264, r=8, lengths=[3, 16, 0, 1]),
    "one_launch_24": dict(K=1032, N=264, r=24, lengths=[16, 0, 3, 1]),
    "one_launch_32": dict(K=1032, N=264, r=32, lengths=[1] * 20),
    "one_launch_32_long": dict(K=4096, N=520, r=32, lengths=[1, 40, 0, 2, 0, 17], ids=[1, 0, 1, -1, 0, 1], n=2),
    "one_launch_64": dict(K=520, N=1032, r=64, lengths=[3, 0, 16, 1]),
    # two launches on 16-row tiles
    "two_launches_8": dict(K=16392, N=136, r=8, lengths=[1, 2, 0, 16]),
    "two_launches_16": dict(K=14336, N=264, r=16, lengths=[1] * 5),
    "two_launches_16_shared": dict(K=8200, N=72, r=16, lengths=[1] * 70, ids=[(7 * i) % 5 - 1 for i in range(70)], n=4),
    "two_launches_32": dict(K=4104, N=136, r=32, lengths=[1, 0, 16, 3]),
    "two_launches_48": dict(K=2736, N=72, r=48, lengths=[5, 30, 0, 0]),
    "two_launches_64": dict(K=2056, N=264, r=64, lengths=[16, 1, 0, 9]),
    "two_launches_72": dict(K=520, N=1032, r=72, lengths=[1, 0, 17, 2]),
    "two_launches_128": dict(K=512, N=136, r=128, lengths=[1, 0, 3, 16]),
    "two_launches_128_wide": dict(K=4104, N=2056, r=128, lengths=[1] * 9, ids=[2, 0, -1, 1, 2, 0, 0, 1, -1], n=3, before=2, after=3),
    # sixteen pieces of the columns, the last one past the end
    "empty_piece": dict(K=8256, N=72, r=16, lengths=[100]),
    "empty_piece_128": dict(K=8256, N=72, r=128, lengths=[50]),
    # a long group among many short ones
    "long_among_short": dict(K=136, N=2048, r=32, lengths=[(5 * i) % 9 if i != 70 else 1500 for i in range(128)]),
    "long_among_short_shared": dict(K=1032, N=264, r=16, lengths=[2] * 150 + [900] + [3] * 49,
                                    ids=[i % 7 - 1 for i in range(200)], n=6),
}


@pytest.mark.parametrize("dtype", [base.F32, base.BF16])
@pytest.mark.parametrize("name", FORMS)
def test_forward(e4b, monkeypatch, name, dtype):
    monkeypatch.setitem(base.CASES, name, FORMS[name])
    base.test_forward(e4b, name, dtype)


@pytest.mark.parametrize("dtype", [base.F32, base.BF16])
@pytest.mark.parametrize("name", FORMS)
def test_backward(e4b, monkeypatch, name, dtype):
    monkeypatch.setitem(base.CASES, name, FORMS[name])
    base.test_backward(e4b, name, dtype)


@pytest.mark.parametrize("name", ["one_launch_32", "two_launches_16_shared", "two_launches_128"])
def test_captured(e4b, name):
    """The decode forms in a captured graph, replayed over changing rows with eager calls in between."""
    p = base.Problem(**FORMS[name])
    y = base._normal(9, p.S, p.N, dtype=base.F32)

    def step():
        return e4b.e4b_grouped_lora(p.x, p.a, p.b, p.scale, p.offsets, p.ids, y=y, z=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(3):
        p.x.copy_(base._normal(30 + i, p.S, p.K))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(captured, step())), i
