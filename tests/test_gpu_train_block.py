"""The example that runs the operators together: a pre-norm MoE block learns
another block's outputs."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_block_learns():
    from grouped_gemm_router_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("train_moe_block", os.path.join(ROOT, "examples", "train_moe_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train(steps=40, T=1024, D=128, F=256, E=4, k=2, lr=0.01)
    # two unrelated blocks: 2 E[silu(z)^2] E[sum of squared gate weights] =
    # 2 * 0.355 * 0.577 for normal z and the two largest of four normal logits;
    # 1024 x 128 outputs of 4 experts leave a few percent
    assert abs(losses[0] / 0.41 - 1) < 0.15
    assert sum(losses[-5:]) < 0.6 * sum(losses[:5])
    again = ex.train(steps=5, T=1024, D=128, F=256, E=4, k=2, lr=0.01)
    assert again == losses[:5]                  # the same bits every time
