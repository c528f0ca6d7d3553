"""Products whose experts' last tiles are short, long or none, at every form: each row and column exactly once."""
import pytest
import torch

from gpu_helpers import DEV
from test_gpu_mxrows import _check, _codes, _offsets

pytestmark = pytest.mark.gpu

# rows of each expert around whole, half and no tiles of 16, 32, 64, 128 and 256 rows
COUNTS = {
    "only short": [1, 3, 8, 2, 5] * 30,
    "only whole": [64] * 70,
    "short and long": [33, 32, 31, 64, 65, 96, 97, 0, 1, 63] * 12,
    "one long, many short": [1500] + [1] * 70 + [0] * 5 + [129, 128, 127, 257, 256, 255],
    "large": [256, 384, 385, 128, 129, 511, 512, 513, 0, 300] * 3,
    "few": [16, 8, 9, 0, 17],
}


@pytest.mark.parametrize("N", [1, 640, 1100])
@pytest.mark.parametrize("name", COUNTS)
def test_every_row_and_column(e4b, name, N):
    counts = COUNTS[name]
    S, E, K = sum(counts) + 3, len(counts), 64
    x, w, off = _codes((S,), K, seed=E), _codes((E, N), K, seed=N), _offsets(counts)
    out = torch.full((S, N), 9.0, device=DEV)
    e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, out=out)
    _check(out, x, w, off, None, K, before=torch.full((S, N), 9.0, device=DEV))


def test_many_rounds_of_large_tiles(e4b):
    """More than twelve tiles of 256 x 256 for each of 256 compute units: one list."""
    counts = COUNTS["large"]
    S, E, N, K = sum(counts) + 3, len(counts), 16650, 32
    x, w, off = _codes((S,), K, seed=E), _codes((E, N), K, seed=N), _offsets(counts)
    out = torch.full((S, N), 9.0, device=DEV)
    e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, out=out)
    _check(out, x, w, off, None, K, before=torch.full((S, N), 9.0, device=DEV))


@pytest.mark.parametrize("S", [40, 3000])
def test_offsets_that_descend_stay_in_bounds(e4b, S):
    """Not a call that the documentation allows: nothing outside the rows is written, and rows of proper groups are whole."""
    N, K, E = 333, 64, 130
    x, w = _codes((S,), K, seed=1), _codes((E, N), K, seed=2)
    room = torch.full((S * N + 1024,), 9.0, device=DEV)
    off = torch.tensor([S, 0] * 65 + [S], dtype=torch.int32, device=DEV)
    e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, out=room[512:512 + S * N].view(S, N))
    torch.cuda.synchronize()
    assert (room[:512] == 9).all() and (room[512 + S * N:] == 9).all()
