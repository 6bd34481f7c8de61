"""The binding of layer norm, Newton-Schulz and Muon without a GPU: what it
needs of torch when it is imported."""
import subprocess
import sys

import pytest

from conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_gemm_router_gb300 import build
    build.build()


def test_import_without_cuda_in_torch():
    """A torch built without CUDA has none of the _cuda functions."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, n)\n"
            "from grouped_gemm_router_gb300 import moe\n"
            "try:\n"
            "    moe.layer_norm_forward(torch.zeros(4, 64), torch.ones(64))\n"
            "except ValueError as e:\n"
            "    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "must be a CUDA tensor" in r.stdout
