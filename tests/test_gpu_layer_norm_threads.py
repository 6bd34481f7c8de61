"""Host threads call the layer norm backward at once, on their own streams, with
widths that share a kernel but not its shared memory size: every call is taken
and has the result that it has alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


@pytest.mark.parametrize("widths", [(8192, 4104), (2048, 1032), (1003, 769)], ids=str)
def test_backward_from_threads(moe, widths):
    T, calls, workers = 8, 20000, 6
    lib, kind = moe.lib, moe.N.MOE_FP32
    errors = []
    start = threading.Barrier(workers)

    def inputs(D):
        g = torch.Generator().manual_seed(D)
        r = lambda *s: torch.randn(*s, generator=g).cuda()
        x, w, ds, dy = r(T, D), r(D), r(T, D), r(T, D).bfloat16()
        f = moe.layer_norm_forward(x, w)
        return dict(dy=dy, x=x, w=w, mean=f["mean"], rstd=f["rstd"], ds=ds)

    sets = {D: inputs(D) for D in widths}
    alone = {D: moe.layer_norm_backward(i["dy"], i["x"], i["w"], i["mean"], i["rstd"], d_stream=i["ds"])
             for D, i in sets.items()}
    outs = []
    for k in range(workers):
        D = widths[k % len(widths)]
        out = {n: torch.full_like(v, float("nan")) for n, v in alone[D].items()}
        scratch = torch.empty(lib.moe_layer_norm_backward_scratch_size(T, D), dtype=torch.uint8, device="cuda")
        outs.append((D, out, scratch, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def worker(k):
        D, out, scratch, stream = outs[k]
        i = sets[D]
        args = (i["dy"].data_ptr(), i["x"].data_ptr(), kind, i["w"].data_ptr(), i["mean"].data_ptr(),
                i["rstd"].data_ptr(), i["ds"].data_ptr(), T, D, out["dx"].data_ptr(), out["dweight"].data_ptr(),
                out["dbias"].data_ptr(), scratch.data_ptr(), scratch.numel(), stream.cuda_stream)
        start.wait()
        call = lib.moe_layer_norm_backward
        for n in range(calls):
            status = call(*args)
            if status:
                errors.append((D, n, status))
                return

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(workers)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for D, out, _, _ in outs:
        assert all(torch.equal(out[n], alone[D][n]) for n in out), D
