"""Which tile form and tile lists a product of MXFP4 rows takes: the library's own rule (csrc/e4b_mx_forms.h, host
arithmetic), compiled by itself.  The other tests' sizes reach the forms they name, every limit has both its sides here, and a
launch has a workgroup for every tile however the rows fall on the experts."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from test_gpu_mx_forms import FORMS
from test_gpu_mx_tile_lists import COUNTS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256
SOURCE = """
#include "e4b_mx_forms.h"
extern "C" void form(long long E, long long N, long long S, int cus, long long* out) {
  const e4b::MxTileForm f = e4b::mx_tile_form(E, N, S, cus);
  const long long blocks = e4b::mx_gemm_blocks(f, E, N, S);
  out[0] = f.bm; out[1] = f.bn; out[2] = f.threads; out[3] = blocks; out[4] = e4b::mx_two_lists(blocks, cus);
}
"""

compiler = next((c for c in ("g++", "clang++", "/opt/rocm/llvm/bin/clang++", "/opt/rocm/bin/hipcc") if shutil.which(c)), None)
pytestmark = pytest.mark.skipif(compiler is None, reason="no C++ compiler")


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    at = tmp_path_factory.mktemp("forms")
    (at / "form.cpp").write_text(SOURCE)
    inc = os.path.join(ROOT, "bit_quantized_mixture_amd", "csrc")
    subprocess.run([compiler, "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + inc, str(at / "form.cpp"), "-o", str(at / "form.so")],
                   check=True)
    call = ctypes.CDLL(str(at / "form.so")).form
    call.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int, ctypes.POINTER(ctypes.c_longlong)]

    def of(S, E, N, cus=CUS):
        """((bm, bn), workgroups, two lists)"""
        out = (ctypes.c_longlong * 5)()
        call(E, N, S, cus, out)
        assert out[2] == (512 if out[0] == 256 else 256)
        return (out[0], out[1]), out[3], bool(out[4])
    return of


def _named(name):
    a, b = name.split(",")[0].split(" x ")
    return int(a), int(b)


@pytest.mark.parametrize("name", FORMS)
def test_sizes_of_the_form_tests(form, name):
    assert form(*FORMS[name])[0] == _named(name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", FORMS)
def test_sizes_of_the_form_tests_on_this_card(form, name):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert form(*FORMS[name], cus=cus)[0] == _named(name), f"{cus} compute units"


# rows, experts, columns on either side of each limit
@pytest.mark.parametrize("under,form_under,over,form_over", [
    # 2048 rows of 8 experts are (2048 + 8 * 255) / 256 = 15 tiles of 256 rows at most: 225 large tiles, and 210
    ((256 * 8, 8, 3840), (256, 256), (256 * 8, 8, 3584), (128, 128)),
    ((96 * 30, 30, 5760), (256, 256), (96 * 30 - 1, 30, 5760), (128, 128)),  # a mean of 96 rows, and of 95
    ((16, 1, 32640), (16, 16), (16, 1, 32641), (64, 128)),             # 255 and 256 tiles of 64 x 128, few rows
    ((16 * 4, 4, 2048), (16, 16), (17 * 4, 4, 2048), (32, 32)),        # a mean of 16 and 17 rows
    ((64, 1, 127 * 32), (16, 16), (64, 1, 128 * 32), (32, 32)),        # 254 and 256 tiles of 32 x 32
    ((64, 1, 320 * 32), (32, 32), (64, 1, 320 * 32 + 1), (64, 64)),    # 640 and 642 of them
    ((64, 1, 256 * 64), (64, 64), (64, 1, 256 * 64 + 1), (128, 128)),  # 256 and 257 tiles of 64 x 64
    ((24 * 8, 8, 28672), (64, 128), (25 * 8, 8, 28672), (128, 128)),   # a mean of 24 and 25 rows
])
def test_both_sides_of_each_limit(form, under, form_under, over, form_over):
    assert form(*under)[0] == form_under and form(*over)[0] == form_over


def test_lists(form):
    """One list from more than twelve workgroups a compute unit on."""
    def large(counts, N):
        f, blocks, two = form(sum(counts) + 3, len(counts), N)
        return f[0] >= 128, two, blocks
    assert large(COUNTS["large"], 1100)[:2] == (True, True) and large(COUNTS["large"], 16650)[:2] == (True, False)
    assert form(8192, 8, 28672)[2] is False and form(8192, 32, 5760)[2] is True
    # 256-row tiles of one expert: 100 and 101 columns of 30 row tiles with 56 and 16 workgroups more than
    S = 30 * 256
    assert form(S, 1, 101 * 256)[1:] == (3046, True) and form(S, 1, 102 * 256)[1:] == (3076, False)


def test_every_tile_has_a_workgroup(form):
    """Workgroup b takes the tiles of XCD b % 8, whose share of either list is an eighth, rounded up where some are
    left: no XCD's share is larger than its workgroups are many."""
    rng = np.random.default_rng(1)
    for _ in range(3000):
        E, S = int(2 ** rng.uniform(0, 8)), int(2 ** rng.uniform(0, 13))
        p = rng.random(E) ** rng.integers(1, 8) + 1e-12
        n = rng.multinomial(S, p / p.sum())
        N = int(2 ** rng.uniform(0, 15))
        (bm, bn), blocks, two = form(S, E, N, int(rng.choice([64, 256, 304])))
        cols, left = -(-N // bn), n % bm
        short = ((left > 0) & (left <= bm // 2)) if two and bm >= 128 else np.zeros(E, dtype=bool)
        whole = int((-(-n // bm) - short).sum()) * cols
        shorts = int(short.sum()) * cols
        for xcd in range(8):
            share = sum(all_ // 8 + (xcd < all_ % 8) for all_ in (whole, shorts))
            assert share <= (blocks - xcd + 7) // 8, (S, E, N, n.tolist())
