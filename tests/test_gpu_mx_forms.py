"""Products of MXFP4 rows at sizes that reach each form of the kernel (tiles of 16 x 16 to 64 x 64 whose waves share
K, of 64 x 128, 128 x 128 and 256 x 256), with every length of K that its loop treats differently, against float64."""
import pytest
import torch

from gpu_helpers import DEV
from test_gpu_mxrows import _check, _codes, _lengths, _normal, _offsets

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# rows, experts, columns (on a card of 256 compute units)
FORMS = {
    "16 x 16": (9, 3, 333),          # few rows an expert, and fewer than 256 tiles of 64 x 128
    "16 x 16, more rows": (75, 2, 70),
    "32 x 32": (190, 2, 1201),       # 256 to 640 tiles of 32 x 32
    "64 x 64": (200, 1, 4061),       # more of those, but no more than 256 tiles of 64 x 64
    "64 x 128": (300, 150, 259),
    "128 x 128": (1200, 30, 645),
    "256 x 256": (6500, 64, 1027),
}
# blocks of 32: fewer than a chunk; a chunk of 8 or 16 and its neighbours; one to nine chunks for the four waves, whole or not
BLOCKS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 90, 127, 144]


@pytest.mark.parametrize("blocks", BLOCKS)
@pytest.mark.parametrize("form", FORMS)
def test_every_length(e4b, form, blocks):
    S, E, N = FORMS[form]
    K = 32 * blocks
    x, w = _codes((S,), K, seed=blocks), _codes((E, N), K, seed=E + N)
    offsets = _offsets(_lengths(S, E, seed=blocks))
    bias = _normal(E, N, seed=9)
    for out_t, b in ((F32, None), (BF16, bias)):
        out = e4b.e4b_grouped_gemm_mxfp4(*x, *w, offsets, bias=b, dtype=out_t)
        _check(out, x, w, offsets, b, K)
        for _ in range(2):
            assert torch.equal(out, e4b.e4b_grouped_gemm_mxfp4(*x, *w, offsets, bias=b, dtype=out_t))


@pytest.mark.parametrize("form", FORMS)
def test_a_nan_byte_in_the_last_block(e4b, form):
    S, E, N = FORMS[form]
    K = 32 * 21
    x, w = _codes((S,), K, seed=1), _codes((E, N), K, seed=2)
    off = _offsets(_lengths(S, E, seed=3))
    clean = e4b.e4b_grouped_gemm_mxfp4(*x, *w, off)
    e = int(torch.nonzero(off[1:] > off[:-1])[0])
    lo, hi = int(off[e]), int(off[e + 1])
    x[1][hi - 1, 20], w[1][e, N - 1, 20] = 255, 255
    out = e4b.e4b_grouped_gemm_mxfp4(*x, *w, off)
    bad = torch.zeros(S, N, dtype=torch.bool, device=DEV)
    bad[hi - 1, :] = True
    bad[lo:hi, N - 1] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("form", FORMS)
def test_rows_around_the_groups_and_behind_the_last_column_stay(e4b, form):
    S, E, N = FORMS[form]
    K = 96
    x, w = _codes((S,), K, seed=1), _codes((E, N), K, seed=2)
    lengths = _lengths(S - 5, E, seed=4)
    off = _offsets(lengths) + 2
    for dt in (F32, BF16):
        room = torch.full((S * N + 512,), 9.0, device=DEV, dtype=dt)
        out = room[:S * N].view(S, N)
        e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, out=out)
        _check(out, x, w, off, None, K, before=torch.full((S, N), 9.0, device=DEV, dtype=dt))
        assert (room[S * N:] == 9).all()
