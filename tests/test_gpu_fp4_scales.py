"""Packed scales of 4-bit weights: the kind that a product takes, their sizes, and numbers at the ends of their ranges."""
import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from test_gpu_fp4 import make_weights, offsets_of, spread
from train_testutil import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_scales_packed_for_the_other_product_are_refused(fmt):
    g = gen(1)
    off = offsets_of([30, 41])
    rows = moe.moe_fp4_quant(spread(g, 71, 64, torch.bfloat16), fmt, off)
    q, tiles, glob, _ = make_weights(g, 2, 128, 64, fmt, gate_up=True)
    q0, plain, glob0, _ = make_weights(gen(2), 2, 128, 64, fmt)
    assert plain.shape == tiles.shape
    fused = (moe.moe_fp4_expert_gemm_silu_mul, moe.moe_fp4_expert_gemm_silu_mul_quant)
    with pytest.raises(ValueError, match="gate_up=False"):
        moe.moe_fp4_expert_gemm(rows, q, tiles, glob)
    for f in fused:
        with pytest.raises(ValueError, match="gate_up=True"):
            f(rows, q0, plain, glob0)
    # the right ones, and tensors that carry no note
    want = moe.moe_fp4_expert_gemm(rows, q0, plain, glob0)
    assert torch.equal(moe.moe_fp4_expert_gemm(rows, q0, plain.clone(), glob0), want)
    h = fused[0](rows, q, tiles, glob)
    assert torch.equal(fused[0](rows, q, tiles.clone(), glob), h)
    fused[1](rows, q, tiles, glob)
