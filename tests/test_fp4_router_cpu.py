"""Refusals of the training router and of the 4-bit rows, weights and products: argument errors are found on the host,
before any device call; and the sizes that the binding works out itself."""
import ctypes
import random

import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from block_fp8_mixture_topk_gb300 import ops

INVALID, SHAPE, WORKSPACE = -1, -2, -3
P = ctypes.c_void_p(0x10000)      # never read: every call below is refused
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
EIGHT = ctypes.c_void_p(0x10008)
NULL = None
BIG = 1 << 40


def call(name, good, **change):
    args = {**good, **change}
    return getattr(ops.lib(), name)(*args.values())


def params(scoring=0, n_group=1, topk_group=1, group_score=0, renormalize=1, scaling=1.0, bias=None):
    return ctypes.byref(ops._RouterParams(scoring, n_group, topk_group, group_score, renormalize, scaling, bias))


def router(**change):
    good = dict(logits=P, ld=64, dtype=0, T=8, E=64, topk=4, params=params(), valid=NULL, ids=P, weights=P, counts=P, tokens=P,
                losses=P, ws=P, wsb=BIG, stream=NULL)
    return call("moe_router", good, **change)


def router_backward(**change):
    good = dict(logits=P, ld=64, dtype=0, T=8, E=64, topk=4, params=params(), ids=P, dweights=P, counts=P, tokens=P, balance=0.1,
                z=0.1, dlogits=P, stream=NULL)
    return call("moe_router_backward", good, **change)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(topk=0), INVALID), (dict(dtype=3), INVALID), (dict(ld=63), INVALID),
    (dict(params=NULL), INVALID), (dict(params=params(scoring=2)), INVALID), (dict(params=params(n_group=0)), INVALID),
    (dict(params=params(group_score=2)), INVALID), (dict(params=params(n_group=4, topk_group=0)), INVALID),
    (dict(params=params(n_group=4, topk_group=5)), INVALID), (dict(logits=NULL), INVALID), (dict(logits=ODD), INVALID),
    (dict(logits=TWO, dtype=2), INVALID), (dict(ids=NULL), INVALID), (dict(ids=TWO), INVALID),
    (dict(topk=33), SHAPE), (dict(topk=65), SHAPE), (dict(E=1025, ld=1025), SHAPE), (dict(params=params(n_group=5, topk_group=1)), SHAPE),
    (dict(params=params(n_group=16, topk_group=1), topk=5), SHAPE), (dict(params=params(n_group=64, topk_group=64)), SHAPE),
])
def test_router_refuses(change, code):
    assert router(**change) == code
    if "n_group=16" not in str(change):
        assert router_backward(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(weights=NULL), INVALID), (dict(weights=TWO), INVALID), (dict(counts=NULL), INVALID), (dict(tokens=NULL), INVALID),
    (dict(losses=NULL), INVALID), (dict(ws=NULL), INVALID), (dict(ws=TWO), INVALID), (dict(wsb=100), WORKSPACE),
    (dict(params=params(bias=0x10002)), INVALID),
])
def test_router_refuses_its_outputs(change, code):
    assert router(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(dweights=NULL), INVALID), (dict(dweights=TWO), INVALID), (dict(dlogits=NULL), INVALID), (dict(dlogits=ODD), INVALID),
    (dict(counts=NULL), INVALID), (dict(tokens=NULL), INVALID), (dict(params=params(scoring=1)), INVALID),
])
def test_router_gradient_refuses(change, code):
    assert router_backward(**change) == code


def test_router_sizes():
    size = ops.lib().moe_router_workspace_size
    assert size(-1, 64) == 0 and size(8, 0) == 0 and size(8, 1025) == 0
    assert size(8, 64) == 8 * (2 * 64 + 2) * 4 and size(10 ** 6, 64) == 152 * (2 * 64 + 2) * 4
    assert router_backward(T=0, logits=NULL) == 0
    update = ops.lib().moe_router_update_bias
    assert update(NULL, P, 8, 0.1, NULL) == INVALID and update(P, NULL, 8, 0.1, NULL) == INVALID
    assert update(P, P, 0, 0.1, NULL) == INVALID and update(P, P, 1025, 0.1, NULL) == SHAPE and update(TWO, P, 8, 0.1, NULL) == INVALID


# ------------------------------------------------------------------------------------------ 4 bits
def quant(**change):
    good = dict(x=P, ldx=128, dtype=0, fmt=0, offsets=P, E=4, rows=10, K=128, codes=P, scales=P, row_scale=NULL, stream=NULL)
    return call("moe_fp4_quant", good, **change)


def dequant(**change):
    good = dict(codes=P, scales=P, row_scale=NULL, fmt=0, offsets=P, E=4, rows=10, K=128, dtype=0, out=P, stream=NULL)
    return call("moe_fp4_dequant", good, **change)


def gemm(**change):
    good = dict(codes=P, scales=P, row_scale=NULL, fmt=0, w=P, w_scales=P, w_global=NULL, offsets=P, rows=10, E=4, N=128, K=128,
                epilogue=0, dtype=0, out=P, out_scales=NULL, stream=NULL)
    return call("moe_fp4_expert_gemm", good, **change)


@pytest.mark.parametrize("change,code", [
    (dict(fmt=2), INVALID), (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(offsets=NULL), INVALID),
    (dict(K=100), SHAPE), (dict(K=32800), SHAPE), (dict(E=1025), SHAPE), (dict(rows=2 ** 31 - 100), SHAPE),
    (dict(codes=NULL), INVALID), (dict(codes=EIGHT), INVALID), (dict(scales=NULL), INVALID), (dict(scales=EIGHT), INVALID),
    (dict(row_scale=P), INVALID), (dict(fmt=1), INVALID), (dict(fmt=1, row_scale=TWO), INVALID),
])
def test_rows_refuse(change, code):
    if "K" in change and change["K"] > 128:
        assert quant(**{**change, "ldx": change["K"]}) == code
    else:
        assert quant(**change) == code
    assert dequant(**change) == code
    assert gemm(**change) == code or (change == dict(fmt=1) and gemm(**change) == INVALID)


@pytest.mark.parametrize("change", [dict(x=NULL), dict(x=ODD), dict(x=TWO, dtype=2), dict(ldx=127), dict(E=0), dict(offsets=NULL, E=1)])
def test_quant_refuses(change):
    assert quant(**change) == INVALID


def test_dequant_refuses():
    assert dequant(out=NULL) == INVALID and dequant(out=EIGHT) == INVALID


@pytest.mark.parametrize("change,code", [
    (dict(epilogue=3), INVALID), (dict(epilogue=1, dtype=2), INVALID), (dict(epilogue=2, dtype=1, out_scales=P), INVALID),
    (dict(epilogue=2), INVALID), (dict(epilogue=0, out_scales=P), INVALID), (dict(epilogue=2, out_scales=EIGHT), INVALID),
    (dict(epilogue=2, out_scales=P, fmt=1, row_scale=P, w_global=P), INVALID), (dict(N=0), INVALID), (dict(E=0), INVALID),
    (dict(offsets=NULL), INVALID), (dict(w=NULL), INVALID), (dict(w=EIGHT), INVALID), (dict(w_scales=NULL), INVALID),
    (dict(w_scales=EIGHT), INVALID), (dict(w_global=P), INVALID), (dict(fmt=1, row_scale=P), INVALID),
    (dict(fmt=1, row_scale=P, w_global=TWO), INVALID), (dict(out=NULL), INVALID), (dict(out=EIGHT), INVALID),
    (dict(N=100), SHAPE), (dict(N=136, epilogue=1), SHAPE), (dict(N=96, epilogue=2, out_scales=P), SHAPE), (dict(N=1 << 24), SHAPE),
    (dict(rows=2 ** 30, N=1 << 20), SHAPE),
])
def test_product_refuses(change, code):
    assert gemm(**change) == code


def test_weights_refuse():
    L = ops.lib()
    assert L.moe_mxfp4_quant_weight(NULL, 0, 2, 8, 64, P, P, NULL) == INVALID
    assert L.moe_mxfp4_quant_weight(EIGHT, 0, 2, 8, 64, P, P, NULL) == INVALID
    assert L.moe_mxfp4_quant_weight(P, 3, 2, 8, 64, P, P, NULL) == INVALID
    assert L.moe_mxfp4_quant_weight(P, 0, -1, 8, 64, P, P, NULL) == INVALID
    assert L.moe_mxfp4_quant_weight(P, 0, 1 << 20, 1 << 20, 64, P, P, NULL) == INVALID
    assert L.moe_mxfp4_quant_weight(P, 0, 2, 8, 60, P, P, NULL) == SHAPE
    assert L.moe_mxfp4_quant_weight(P, 0, 0, 8, 64, P, P, NULL) == 0
    assert L.moe_fp4_pack_scales(NULL, 0, 2, 8, 64, 0, P, NULL) == INVALID
    assert L.moe_fp4_pack_scales(P, 0, 2, 8, 64, 0, EIGHT, NULL) == INVALID
    assert L.moe_fp4_pack_scales(P, 2, 2, 8, 64, 0, P, NULL) == INVALID
    assert L.moe_fp4_pack_scales(P, 0, 0, 8, 64, 0, P, NULL) == INVALID
    assert L.moe_fp4_pack_scales(P, 0, 2, 40, 64, 1, P, NULL) == SHAPE
    assert L.moe_fp4_pack_scales(P, 0, 2, 8, 60, 0, P, NULL) == SHAPE


def test_sizes_of_scales():
    """The binding's own sums are the library's, and no two experts' rows share a tile."""
    L, r = ops.lib(), random.Random(1)
    for _ in range(500):
        f, n, E, K = (r.randint(0, 1), r.choice([0, 1, 223, 224, 225, r.randint(0, 2 ** 31)]), r.choice([0, 1, 7, 1024, 1025]),
                      r.choice([0, 32, 64, 100, 256, 288, 32768, 32800]))
        assert L.moe_fp4_row_scale_bytes(f, n, E, K) == ops._fp4_row_scale_bytes(f, n, E, K)
        N = r.randint(1, 40000)
        if K and K % 32 == 0 and E:
            assert L.moe_fp4_weight_scale_bytes(f, E, N, K) == ops._fp4_weight_scale_bytes(f, E, N, K)
    for _ in range(200):
        counts = [r.choice([0, 1, 223, 224, 225, r.randint(0, 2000)]) for _ in range(r.randint(1, 40))]
        o, last = 0, -1
        for e, c in enumerate(counts + [r.randint(0, 500)]):     # the last: rows of no expert
            if c:
                first = o // 224 + e
                assert first > last
                last = first + (c - 1) // 224
            o += c
        assert last < o // 224 + len(counts) + 1


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (lambda: moe.moe_fp4_quant(x), lambda: moe.moe_mxfp4_quant_weight(x[None]), lambda: moe.moe_router(x, 2),
              lambda: moe.moe_fp4_pack_scales(torch.zeros(1, 4, 2, dtype=torch.uint8)),
              lambda: moe.moe_router_update_bias(torch.zeros(4), torch.zeros(4, dtype=torch.int32), 0.1)):
        with pytest.raises(ValueError):
            f()
    rows = moe.Fp4Rows(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8), None, "mxfp4", None)
    with pytest.raises(ValueError):
        moe.moe_fp4_dequant(rows)
    with pytest.raises(ValueError, match="format"):
        moe.moe_fp4_dequant(rows._replace(format="fp4"))
