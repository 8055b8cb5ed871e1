"""The router, the movement of the rows and the 4-bit experts together, as a layer uses them, and the examples on them."""
import os
import sys

import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from test_gpu_fp4 import quantise64, weights64
from train_testutil import gen, status, status_clear

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serve_fp4_block as serve  # noqa: E402
import train_moe_block as train  # noqa: E402

pytestmark = pytest.mark.gpu


def reference(p, fmt, x, ids, weights):
    """The block in 64 bits on the numbers that the 4-bit weights stand for, h rounded to bf16 and in 4 bits as the layer's."""
    def numbers(name):
        if fmt == "mxfp4":
            codes, scales = moe.moe_mxfp4_quant_weight(p[name])
            return weights64(codes, scales, None, fmt)
        return weights64(*moe.moe_nvfp4_quant_weight(p[name]), fmt)
    w13, w2 = numbers("w13"), numbers("w2")
    rows = quantise64(x, fmt).to(x.device)
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(w13.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            gate, up = (rows[t] @ w13[e].T).chunk(2, 1)
            h = quantise64((torch.nn.functional.silu(gate) * up).to(torch.bfloat16), fmt).to(x.device)
            out.index_add_(0, t, (h @ w2[e].T) * weights[t, j][:, None].double())
    return out


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 32, 8, 2), (300, 128, 96, 8, 2), (77, 256, 160, 33, 5), (2000, 320, 512, 16, 4)])
def test_block(T, H, I, E, k, fmt):
    p = serve.weights(H, I, E, seed=T)
    q = serve.load(p, fmt)
    x = torch.randn(T, H, generator=gen(T)).bfloat16().cuda()
    status_clear()
    out = serve.forward(q, x, k)
    route = moe.moe_router(x.float() @ q["router"].T, k)
    want = reference(p, fmt, x, route.ids, route.weights)
    # y and out are rounded to bf16, 2^-9 of their size in the mean square at most.  An fp32 sum a few 2^-22 off takes h over
    # a border of bf16 (one value in 2^13: 2^-8 of its size) and that over one of 4 bits (a step, at most half of the value: as
    # rarely, one in 2^13, of the values near the border only): below 2^-8 of the result's size in the mean square together
    assert ((out.double() - want).norm() / want.norm()).item() < 2 * 2.0 ** -9 + 2.0 ** -8
    assert status() == 0


def test_padded_tokens_cost_nothing():
    """Tokens that the router leaves out send no rows, and come back as zero."""
    p = serve.weights(128, 64, 8)
    q = serve.load(p, "mxfp4")
    x = torch.randn(100, 128, generator=gen(1)).bfloat16().cuda()
    valid = torch.arange(100, device="cuda") < 60
    x[60:] = float("nan")
    route = moe.moe_router(torch.nan_to_num(x.float()) @ q["router"].T, 2, valid=valid, losses=True)
    d = moe.moe_dispatch(x, route.ids, 8)
    rows = moe.moe_fp4_quant(d.rows, "mxfp4", d.expert_offsets)
    act = moe.moe_fp4_expert_gemm_silu_mul_quant(rows, *q["w13"])
    out = moe.moe_combine(moe.moe_fp4_expert_gemm(act, *q["w2"]), d.pos, route.weights)
    assert int(route.counts.sum()) == 120 and int(route.tokens) == 60
    assert (out[60:] == 0).all() and torch.equal(out[:60], serve.forward(q, x[:60].contiguous(), 2))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_serving_example_runs(fmt):
    off = serve.main(["--tokens", "300", "--hidden", "256", "--inter", "96", "--experts", "16", "--topk", "4", "--steps", "2",
                      "--format", fmt])
    assert 0.0 < off < 0.5


def test_training_example_with_losses():
    """The gradients of the block with the balance and z losses, against differences along the gradient itself."""
    T, H, I, E, k = 200, 64, 32, 8, 2
    p = train.init_params(H, I, E, seed=5)
    x = torch.randn(T, H, generator=gen(6)).bfloat16().cuda()
    zero = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    _, s = train.forward(p, x, k, losses=True)
    g = train.backward(p, s, zero, balance=1.0, z=0.5)["router"]
    l = s["logits"].double().requires_grad_()
    share, f = torch.softmax(l, 1), s["route"].counts.double() * E / (k * T)
    loss = (f * share.mean(0)).sum() + 0.5 * torch.logsumexp(l, 1).square().mean()
    want = torch.autograd.grad(loss, l)[0].T @ s["h"].double()
    # fp32 logits' gradients, an fp32 product over 200 tokens
    assert ((g.double() - want).norm() / want.norm()).item() < 1e-5
    losses = train.main(["--tokens", "64", "--hidden", "64", "--inter", "32", "--experts", "8", "--topk", "2", "--steps", "2",
                         "--balance", "0.01", "--z", "0.001"])
    assert len(losses) == 2


def test_bindings_refuse():
    x = torch.randn(6, 64, device="cuda").bfloat16()
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    rows = moe.moe_fp4_quant(x, "nvfp4", off)
    q, s, total = moe.moe_nvfp4_quant_weight(torch.randn(2, 32, 64, device="cuda").bfloat16())
    tiles = moe.moe_fp4_pack_scales(s, "nvfp4")
    good = (rows, q, tiles, total)
    moe.moe_fp4_expert_gemm(*good)
    for bad, error in (((rows, q[:1], tiles, total), ValueError), ((rows, q, tiles[:1], total), ValueError),
                       ((rows, q, tiles, None), ValueError), ((rows, q, tiles, total[:1]), ValueError),
                       ((rows, q.float(), tiles, total), TypeError), ((rows._replace(row_scale=None), q, tiles, total), ValueError),
                       ((rows._replace(scales=rows.scales[:-1]), q, tiles, total), ValueError),
                       ((rows._replace(format="mxfp4"), q, tiles, total), ValueError),
                       ((rows._replace(expert_offsets=off[:2]), q, tiles, total), ValueError),
                       ((rows, q[:, :, :16].contiguous(), tiles, total), ValueError), ((rows, q.cpu(), tiles, total), ValueError)):
        with pytest.raises(error):
            moe.moe_fp4_expert_gemm(*bad)
    with pytest.raises(TypeError):
        moe.moe_fp4_expert_gemm_silu_mul(*good, dtype=torch.float32)
    with pytest.raises(ValueError):
        moe.moe_fp4_expert_gemm_silu_mul_quant(*good)          # 32 rows: I = 16 is no group of 32
    with pytest.raises(ValueError):
        moe.moe_fp4_quant(x, "nvfp4", off[::2])
    with pytest.raises(moe.MoeError):
        moe.moe_fp4_quant(x[:, :48].contiguous())
    for change, error in ((dict(topk=0), ValueError), (dict(topk=65), moe.MoeError), (dict(group_score="sum"), ValueError),
                          (dict(valid=torch.ones(5, dtype=torch.bool, device="cuda")), ValueError),
                          (dict(valid=torch.ones(6, device="cuda")), TypeError),
                          (dict(routing=moe.RoutingParams(bias=torch.zeros(63, device="cuda"))), ValueError)):
        with pytest.raises(error):
            moe.moe_router(x, **{"topk": 2, **change})
    r = moe.moe_router(x, 2)
    dw = torch.zeros(6, 2, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_router_backward(x, r, dw, balance_coef=0.1)     # no loads were asked for
    r = moe.moe_router(x, 2, losses=True, routing=moe.RoutingParams("sigmoid"))
    with pytest.raises(ValueError):
        moe.moe_router_backward(x, r, dw, routing=moe.RoutingParams("sigmoid"), z_coef=0.1)
    with pytest.raises(ValueError):
        moe.moe_router_backward(x, r, dw[:5])
    with pytest.warns(UserWarning, match="autograd"):
        moe.moe_router(x.float().requires_grad_(), 2)
    with pytest.warns(UserWarning, match="autograd"):
        moe.moe_fp4_quant(x.requires_grad_())


def test_empty():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for fmt in ("mxfp4", "nvfp4"):
        rows = moe.moe_fp4_quant(x, fmt, off)
        assert moe.moe_fp4_dequant(rows).shape == (0, 64)
        w = torch.randn(2, 64, 64, device="cuda").bfloat16()
        if fmt == "mxfp4":
            (q, s), total = moe.moe_mxfp4_quant_weight(w), None
        else:
            q, s, total = moe.moe_nvfp4_quant_weight(w)
        assert moe.moe_fp4_expert_gemm(rows, q, moe.moe_fp4_pack_scales(s, fmt), total).shape == (0, 64)
        h = moe.moe_fp4_expert_gemm_silu_mul_quant(rows, q, moe.moe_fp4_pack_scales(s, fmt, True), total)
        assert h.codes.shape == (0, 16)
