"""Buffer stores of more than 64 bits take their offset from a vector register.  A store reads its
data registers some cycles after it is issued: the next instructions may not write them.  The
compiler keeps that distance for every form of wide store but one, the buffer store whose offset is
in a scalar register, and there rows came out with the next value of a register in them.  No GPU needed."""
import importlib.util
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_mixture_amd", "csrc")
WIDE = re.compile(r"\bbuffer_store_dwordx[34] v\[[0-9:]+\], (?:v\d+|off), s\[[0-9:]+\], (?:s\d+|m0|vcc\w*|ttmp\d+)\b")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")


def _sources():
    return [f for f in sorted(os.listdir(CSRC)) if f.endswith(".hip")
            and "raw_buffer_store" in open(os.path.join(CSRC, f)).read()]


def test_the_pattern_knows_the_form():
    assert WIDE.search("\tbuffer_store_dwordx4 v[82:85], v116, s[8:11], s48 offen nt")
    assert not WIDE.search("\tbuffer_store_dwordx4 v[82:85], v116, s[8:11], 0 offen nt")
    assert not WIDE.search("\tbuffer_store_dwordx2 v[82:83], v116, s[8:11], s48 offen nt")


@pytest.mark.parametrize("source", _sources())
def test_wide_buffer_stores_have_no_scalar_offset(source, tmp_path):
    spec = importlib.util.spec_from_file_location("e4b_build", os.path.join(ROOT, "bit_quantized_mixture_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    flags = [f for f in build.compile_cmd("x")[1:] if f not in ("-shared", "-o", "x") and not f.endswith(".hip")]
    out = str(tmp_path / "k.s")
    subprocess.run([build.hipcc(), *flags, "--cuda-device-only", "-S", os.path.join(CSRC, source), "-o", out],
                   check=True, capture_output=True)
    text = open(out).read()
    assert "buffer_store" in text
    assert WIDE.findall(text) == []
