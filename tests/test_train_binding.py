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


class FakeCuda:
    """What the checks look at of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        import torch
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        raise AssertionError("used before all tensors were checked")


def _calls(moe, other, which):
    """The calls, tensor number `which` of each on device `other`."""
    import torch
    bf, f = torch.bfloat16, torch.float32

    def make(*specs):
        return [FakeCuda(s, t, other if i == which else 0) for i, (s, t) in enumerate(specs)]

    x, w, b, add, y = make(((4, 64), bf), ((64,), f), ((64,), f), ((4, 64), bf), ((4, 64), bf))
    yield 5, lambda: moe.layer_norm_forward(x, w, bias=b, add=add, y=y)
    dy, x1, w1, mu, r, ds = make(((4, 64), bf), ((4, 64), bf), ((64,), f), ((4,), f), ((4,), f), ((4, 64), bf))
    yield 6, lambda: moe.layer_norm_backward(dy, x1, w1, mu, r, d_stream=ds)
    g, out, ws = make(((2, 64, 64), f), ((2, 64, 64), bf), ((1 << 20,), torch.uint8))
    yield 3, lambda: moe.newton_schulz(g, out=out, workspace=ws)
    wt, g2, m, low, wsp = make(((2, 64, 64), f), ((2, 64, 64), f), ((2, 64, 64), f), ((2, 64, 64), bf), ((1 << 20,), torch.uint8))
    yield 5, lambda: moe.muon_step([wt], [g2], [m], lr=0.1, weights_bf16=[low], workspace=wsp)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """One tensor elsewhere, and all of them on a device that is not the current one."""
    import torch
    from grouped_gemm_router_gb300 import moe
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: (_ for _ in ()).throw(AssertionError("launched")))
    for which in range(6):
        for n, call in _calls(moe, 1, which):
            if which < n:
                with pytest.raises(ValueError, match="cuda:1|cuda:0"):
                    call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for _, call in _calls(moe, 1, 99):
        with pytest.raises(ValueError, match="current device"):
            call()
