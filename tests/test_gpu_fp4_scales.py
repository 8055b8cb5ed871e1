"""Scales of 4-bit numbers: the kind that a product takes, and quotients of 16-bit rows as near to a border as they come."""
import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from test_gpu_fp4 import make_weights, offsets_of, quantise64, same, spread
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


def test_nearest_quotients_of_fp16_rows():
    """x * 2688 / (b m) of an fp16 row with largest m and a group's e4m3 scale b, next to a border h between codes: x = 1584 with
    m = 2047, b = 13 (as significands) is 2^-17 of itself from 1.25, the nearest that there is; and all the others near it."""
    near = []
    for m in range(1024, 2048):
        for b in range(8, 16):
            for h in (1, 3, 5, 7):
                v = h * b * m                          # 21 x against it, both up to a power of two
                while v < 21 * 1024:
                    v *= 2
                shift = 0
                while v >= 21 * 2048 << shift:
                    shift += 1
                x = round(v / (21 << shift))
                off = abs((21 * x << shift) - v)
                if off and off / v < 2.0 ** -15.5 and 1024 <= x < 2048:
                    near.append((off / v, m, b, h, x))
    near.sort()
    assert near[0][0] == 1 / (65 * 2047) and near[0][1:] == (2047, 13, 5, 1584)
    rows = []
    for _, m, b, h, x in near:
        # groups whose largest makes the scale b 2^q (448 is the row's largest), with x among them at powers of two
        r = torch.zeros(32, 16, dtype=torch.float64)
        r[0, 0] = m / 1024
        for i in range(1, 32):
            r[i, 0] = b * 2.0 ** (4 - i // 3) / 448 * (m / 1024)
            for j in range(1, 16):
                v = x / 1024 * 2.0 ** -(j - 1)
                r[i, j] = v if v <= r[i, 0] else 0.0
        rows.append(r.reshape(512))
    x = torch.stack(rows).half().cuda()
    got = moe.moe_fp4_dequant(moe.moe_fp4_quant(x, "nvfp4"), torch.float32)
    same(got, quantise64(x, "nvfp4"), "values")


@pytest.mark.parametrize("top", [2047, 2046, 1985, 1625, 1025, 1024])
def test_borders_of_fp16_rows_with_the_longest_significands(top):
    """Every fp16 number up to eight powers of two below the row's largest."""
    below = (1 + torch.arange(1024, dtype=torch.float64) / 1024)[None] * 2.0 ** -torch.arange(0, 8)[:, None]
    v = below.reshape(-1)
    v = v[v <= top / 1024]
    x = torch.cat([v, torch.zeros(-len(v) % 64 + 64)])
    x[-1] = top / 1024
    x = torch.stack([x, -x.flip(0)]).half().cuda()
    same(moe.moe_fp4_dequant(moe.moe_fp4_quant(x, "nvfp4"), torch.float32), quantise64(x, "nvfp4"), f"{top}")
