"""The token and adapter kernels spill no registers (the compiler's own report; no GPU needed)."""
import importlib.util
import os
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")


@pytest.mark.parametrize("source,kernels", [
    ("tokens.hip", ["permute_kernel", "permute_scatter_kernel", "combine_rows_kernel", "combine_backward_kernel"]),
    ("lora.hip", ["shrink_kernel", "expand_kernel", "fused_kernel", "grad_kernel", "between_kernel", "grad_reduce_kernel"])])
def test_no_spills(source, kernels):
    spec = importlib.util.spec_from_file_location("e4b_build", os.path.join(ROOT, "bit_quantized_mixture_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    usage = build.resource_usage(source)
    for k in kernels:
        assert any(k in name for name in usage), k
    assert not {name: u for name, u in usage.items() if u.get("vgpr_spill") or u.get("scratch")}
