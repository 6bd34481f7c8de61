"""What the C ABI allows of overlap: the forward's h may be x itself, the
backward's dx may be d_stream itself.  The results are those of separate
buffers, bit for bit, whatever form of the kernel a width takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SIZES = [(300, 128), (300, 768), (64, 1005), (64, 1008), (33, 2048), (20, 4096), (12, 8192), (12, 8191), (5000, 768)]


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_in_place(moe, T, D, dtype):
    lib, kind = moe.lib, moe.N.MOE_FP32 if dtype == torch.float32 else moe.N.MOE_BF16
    g = torch.Generator(device="cuda").manual_seed(T + D)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    x, w, b, add, dy, ds = r(T, D).to(dtype), r(D), r(D), r(T, D).bfloat16(), r(T, D).bfloat16(), r(T, D).to(dtype)
    ref = moe.layer_norm_forward(x, w, bias=b, add=add)
    h, y, mean, rstd = x.clone(), torch.empty_like(add), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    assert lib.moe_layer_norm_forward(h.data_ptr(), kind, add.data_ptr(), w.data_ptr(), b.data_ptr(), 1e-5, T, D,
                                      y.data_ptr(), h.data_ptr(), mean.data_ptr(), rstd.data_ptr(), stream) == 0
    assert torch.equal(h, ref["h"]) and torch.equal(y, ref["y"])
    assert torch.equal(mean, ref["mean"]) and torch.equal(rstd, ref["rstd"])
    gref = moe.layer_norm_backward(dy, h, w, mean, rstd, d_stream=ds)
    d, dw, db = ds.clone(), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    scratch = torch.empty(lib.moe_layer_norm_backward_scratch_size(T, D), dtype=torch.uint8, device="cuda")
    assert lib.moe_layer_norm_backward(dy.data_ptr(), h.data_ptr(), kind, w.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                       d.data_ptr(), T, D, d.data_ptr(), dw.data_ptr(), db.data_ptr(),
                                       scratch.data_ptr(), scratch.numel(), stream) == 0
    assert torch.equal(d, gref["dx"]) and torch.equal(dw, gref["dweight"]) and torch.equal(db, gref["dbias"])
