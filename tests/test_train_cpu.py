"""The training operators' refusals: argument errors are found on the host, before any device call."""
import ctypes

import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from block_fp8_mixture_topk_gb300 import ops

INVALID, SHAPE, WORKSPACE = -1, -2, -3
P = ctypes.c_void_p(0x10000)      # never read: every call below is refused
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)    # on a 16-bit element, not on 16 bytes
NULL = None
BIG = 1 << 40


def call(name, good, **change):
    args = {**good, **change}
    return getattr(ops.lib(), name)(*args.values())


def dispatch(**change):
    good = dict(x=P, ldx=64, dtype=0, ids=P, T=8, topk=2, E=4, H=64, rows=P, offsets=P, pair_ids=P, pos=P, ws=P,
                wsb=BIG, stream=NULL)
    return call("moe_dispatch", good, **change)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(topk=0), INVALID), (dict(E=0), INVALID), (dict(H=0), INVALID), (dict(ldx=63), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(x=NULL), INVALID), (dict(ids=NULL), INVALID),
    (dict(rows=NULL), INVALID), (dict(offsets=NULL), INVALID), (dict(pair_ids=NULL), INVALID), (dict(pos=NULL), INVALID),
    (dict(x=ODD), INVALID), (dict(rows=ODD), INVALID), (dict(x=TWO, dtype=2), INVALID),
    (dict(topk=33), SHAPE), (dict(E=1025), SHAPE), (dict(H=65537, ldx=65537), SHAPE), (dict(T=2 ** 30, topk=2), SHAPE),
    (dict(T=300000, wsb=0), WORKSPACE), (dict(T=300000, ws=NULL), INVALID),
])
def test_dispatch_refuses(change, code):
    assert dispatch(**change) == code


def test_dispatch_workspace_size():
    size = ops.lib().moe_dispatch_workspace_size
    assert size(8, 2, 64) == 0 and size(300000, 2, 64) > 0       # few pairs are counted in the one launch
    assert size(-1, 2, 64) == 0 and size(0, 2, 64) == 0


def combine(**change):
    good = dict(y=P, ldy=64, dtype=0, pos=P, weights=P, T=8, topk=2, H=64, rows=16, out=P, stream=NULL)
    return call("moe_combine", good, **change)


def combine_backward(**change):
    good = dict(dout=P, ldo=64, y=P, ldy=64, dtype=0, pos=P, pair_ids=P, weights=P, T=8, topk=2, H=64, rows=16, dy=P,
                dw=P, stream=NULL)
    return call("moe_combine_backward", good, **change)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(topk=0), INVALID), (dict(H=0), INVALID), (dict(ldy=63), INVALID), (dict(dtype=9), INVALID),
    (dict(rows=-1), INVALID), (dict(y=NULL), INVALID), (dict(pos=NULL), INVALID), (dict(y=ODD), INVALID),
    (dict(topk=33), SHAPE), (dict(rows=2 ** 31), SHAPE), (dict(H=65537, ldy=65537), SHAPE),
])
def test_combine_refuses(change, code):
    assert combine(**change) == code
    if "H" in change:
        change = {**change, **({"ldo": 65537} if change["H"] > 64 else {})}
    assert combine_backward(**change) == code


def test_combine_refuses_its_outputs():
    assert combine(out=NULL) == INVALID and combine(out=ODD) == INVALID
    for change in (dict(dy=NULL), dict(dw=NULL), dict(dout=NULL), dict(pair_ids=NULL), dict(ldo=63), dict(dy=ODD),
                   dict(dout=ODD)):
        assert combine_backward(**change) == INVALID
    assert combine(T=0) == 0


def test_token_binding_refuses():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: moe.moe_dispatch(x, ids, 3), lambda: moe.moe_combine(x, ids),
              lambda: moe.moe_dispatch_backward(x, ids), lambda: moe.moe_combine_backward(x, x, ids, ids[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            f()
