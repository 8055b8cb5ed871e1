"""The training operators' refusals: argument errors are found on the host, before any device call."""
import ctypes
import importlib.util
import sys
import warnings

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


def pre_norm(**change):
    good = dict(x=P, ldx=64, dtype=0, w=P, wt=2, off=0.0, eps=1e-6, T=8, H=64, h=P, rstd=P, stream=NULL)
    return call("moe_pre_norm", good, **change)


def pre_norm_backward(**change):
    good = dict(dh=P, ldd=64, x=P, ldx=64, dtype=0, w=P, wt=2, off=0.0, rstd=P, dres=P, ldr=64, T=8, H=64, dx=P, dw=P,
                ws=P, wsb=BIG, stream=NULL)
    return call("moe_pre_norm_backward", good, **change)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(ldx=63), INVALID), (dict(dtype=3), INVALID), (dict(wt=3), INVALID),
    (dict(x=NULL), INVALID), (dict(w=NULL), INVALID), (dict(rstd=NULL), INVALID), (dict(x=ODD), INVALID),
    (dict(w=TWO), INVALID), (dict(H=16385, ldx=16385), SHAPE),
])
def test_pre_norm_refuses(change, code):
    assert pre_norm(**change) == code
    assert pre_norm_backward(**change) == code


def test_pre_norm_refuses_its_outputs():
    assert pre_norm(h=NULL) == INVALID and pre_norm(h=ODD) == INVALID
    for change in (dict(dx=NULL), dict(dw=NULL), dict(dh=NULL), dict(ldd=63), dict(ldr=63), dict(dx=ODD), dict(ws=NULL)):
        assert pre_norm_backward(**change) == INVALID
    assert pre_norm_backward(wsb=0) == WORKSPACE
    assert ops.lib().moe_norm_backward_workspace_size(0, 64) == 0
    assert ops.lib().moe_norm_backward_workspace_size(4096, 64) > 0


def params(**change):
    good = dict(weight=0x10000, next_weight=0, gate=0x10000, gate_stride=64, weight_dtype=2, gate_kind=3, gate_sigmoid=0,
                weight_offset=0.0, eps=1e-6, residual_scale=1.0, block_scale=1.0)
    return ctypes.byref(ops._PostNormParams(*{**good, **change}.values()))


def post_norm(prm=None, **change):
    good = dict(y=P, ldy=64, r=P, ldr=64, dtype=0, prm=params(**(prm or {})), T=8, H=64, out=P, rstd=P, h2=P, r2=P,
                stream=NULL)
    return call("moe_post_norm", good, **change)


def post_norm_backward(prm=None, **change):
    good = dict(dout=P, ldo=64, y=P, ldy=64, dtype=0, prm=params(**(prm or {})), rstd=P, T=8, H=64, dy=P, dres=P, dgate=P,
                dw=P, ws=P, wsb=BIG, stream=NULL)
    return call("moe_post_norm_backward", good, **change)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(ldy=63), INVALID), (dict(dtype=3), INVALID), (dict(y=NULL), INVALID),
    (dict(rstd=NULL), INVALID), (dict(y=ODD), INVALID), (dict(H=16385, ldy=16385), SHAPE),
])
def test_post_norm_refuses(change, code):
    assert post_norm(**change) == code
    assert post_norm_backward(**change) == code


@pytest.mark.parametrize("prm", [
    dict(weight=0), dict(weight=0x10002), dict(weight_dtype=5), dict(gate_kind=4), dict(gate_kind=-1), dict(gate_kind=0),
    dict(gate=0), dict(gate_stride=63), dict(gate_kind=1, gate_stride=0), dict(gate=0x10001),
])
def test_post_norm_refuses_parameters(prm):
    assert post_norm(prm) == INVALID
    assert post_norm_backward(prm) == INVALID


def test_post_norm_refuses_its_outputs():
    nxt = dict(next_weight=0x10000)
    assert call("moe_post_norm", dict(y=P, ldy=64, r=P, ldr=64, dtype=0, prm=NULL, T=8, H=64, out=P, rstd=P, h2=P, r2=P,
                                      stream=NULL)) == INVALID
    assert post_norm(out=NULL) == INVALID and post_norm(r=NULL) == INVALID and post_norm(ldr=63) == INVALID
    assert post_norm(nxt, h2=NULL) == INVALID and post_norm(nxt, r2=NULL) == INVALID
    for change in (dict(dy=NULL), dict(dw=NULL), dict(dout=NULL), dict(ldo=63), dict(dres=ODD), dict(ws=NULL)):
        assert post_norm_backward(**change) == INVALID
    assert post_norm_backward(dict(gate=0, gate_kind=0)) == INVALID      # a gradient for no gate
    assert post_norm_backward(wsb=8) == WORKSPACE


def test_norm_binding_refuses():
    x = torch.zeros(4, 8)
    for f in (lambda: moe.moe_pre_norm(x, x[0]), lambda: moe.moe_post_norm(x, x, x[0]),
              lambda: moe.moe_pre_norm_backward(x, x, x[0], x[:, 0]), lambda: moe.moe_post_norm_backward(x, x, x[0], x[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def clip(n=2, grads=(0x10000, 0x20000), out=None, numel=(4, 5), dtype=(0, 2), kind=0, limit=1.0, eps=1e-6, total=P, ws=P,
         wsb=BIG):
    a = (ctypes.c_void_p * 2)(*grads)
    o = (ctypes.c_void_p * 2)(*(out or grads))
    return ops.lib().moe_clip_grads(a, o, (ctypes.c_int64 * 2)(*numel), (ctypes.c_int32 * 2)(*dtype), n, kind, limit, eps,
                                    total, ws, wsb, None)


@pytest.mark.parametrize("change,code", [
    (dict(n=-1), INVALID), (dict(kind=2), INVALID), (dict(limit=-1.0), INVALID), (dict(limit=float("nan")), INVALID),
    (dict(eps=-1.0), INVALID), (dict(total=NULL), INVALID), (dict(numel=(4, -1)), INVALID), (dict(dtype=(0, 3)), INVALID),
    (dict(grads=(0x10000, 0)), INVALID), (dict(grads=(0x10001, 0x20000)), INVALID), (dict(out=(0x10000, 0x20002)), INVALID),
    (dict(numel=(1 << 51, 1)), SHAPE), (dict(wsb=0), WORKSPACE), (dict(ws=NULL), INVALID),
])
def test_clip_refuses(change, code):
    assert clip(**change) == code


def test_clip_binding_refuses():
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_clip_grads([torch.zeros(3)], 1.0)
    with pytest.raises(ValueError, match="norm_type"):
        moe.moe_clip_grads([], 1.0, norm_type=1)
    with pytest.raises(ValueError, match="one tensor per gradient"):
        moe.moe_clip_grads([torch.zeros(3)], 1.0, out=[])


def product(**change):
    good = dict(a=P, lda=64, dtype=0, w=P, off=P, rows=16, E=4, N=32, K=64, epilogue=1, out=P, gu=P, stream=NULL)
    return call("moe_expert_gemm", good, **change)


def dgrad(**change):
    good = dict(dc=P, ldd=32, dtype=0, w=P, off=P, rows=16, E=4, N=32, K=64, gu=P, ldgu=128, out=P, stream=NULL)
    return call("moe_expert_gemm_dgrad", good, **change)


def wgrad(**change):
    good = dict(dc=P, ldd=32, a=P, lda=64, dtype=0, off=P, rows=16, E=4, N=32, K=64, dw=P, stream=NULL)
    return call("moe_expert_gemm_wgrad", good, **change)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=-1), INVALID), (dict(off=NULL), INVALID), (dict(E=1025), SHAPE), (dict(N=12), SHAPE), (dict(K=60), SHAPE),
    (dict(rows=2 ** 31), SHAPE),
])
def test_products_refuse(change, code):
    for f in (product, dgrad, wgrad):
        assert f(**change) == code


def test_products_refuse_operands():
    for change, code in ((dict(a=NULL), INVALID), (dict(w=NULL), INVALID), (dict(out=NULL), INVALID), (dict(lda=56), INVALID),
                         (dict(lda=65), SHAPE), (dict(a=TWO), INVALID), (dict(w=TWO), INVALID), (dict(out=TWO), INVALID),
                         (dict(gu=TWO), INVALID), (dict(epilogue=2), INVALID), (dict(epilogue=0), INVALID), (dict(N=40), SHAPE)):
        assert product(**change) == code, change
    for change, code in ((dict(dc=NULL), INVALID), (dict(w=NULL), INVALID), (dict(out=NULL), INVALID), (dict(ldd=24), INVALID),
                         (dict(ldd=33), SHAPE), (dict(ldgu=120), INVALID), (dict(ldgu=129), SHAPE), (dict(gu=TWO), INVALID)):
        assert dgrad(**change) == code, change
    for change, code in ((dict(dc=NULL), INVALID), (dict(a=NULL), INVALID), (dict(dw=NULL), INVALID), (dict(ldd=24), INVALID),
                         (dict(lda=56), INVALID), (dict(lda=65), SHAPE), (dict(ldd=33), SHAPE), (dict(dw=TWO), INVALID)):
        assert wgrad(**change) == code, change


def test_expert_binding_refuses():
    x, off = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    for f in (lambda: moe.moe_expert_gemm(x, w, off), lambda: moe.moe_expert_gemm_silu_mul(x, w, off),
              lambda: moe.moe_expert_gemm_dgrad(x, w, off), lambda: moe.moe_expert_gemm_wgrad(x, x, off)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.mark.parametrize("kind", [1, 3])
def test_post_norm_of_no_rows_needs_no_gate(kind):
    """An empty tensor's address is 0: a gate of no values has none.  (A row or a channel gate still needs one.)"""
    empty = dict(gate=0, gate_kind=kind)
    assert post_norm(empty, T=0, y=NULL, r=NULL, out=NULL, rstd=NULL) == 0
    assert post_norm(empty, T=1) == INVALID and post_norm_backward(empty, T=1) == INVALID
    assert post_norm(dict(gate=0, gate_kind=2), T=0) == INVALID
    assert post_norm_backward(dict(gate=0, gate_kind=2), T=0) == INVALID
    assert post_norm_backward(dict(gate=0, gate_kind=0), T=0) == INVALID    # a gradient for no gate


class OnDevice:
    """What the binding asks of a dense CUDA tensor before it launches."""
    is_cuda = True
    requires_grad = False

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.device = dtype, shape, torch.device("cuda", device)

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


def device_calls():
    """(function, keyword operands) of every training operator, each operand in order of shape and type."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, rows, vec, t = (bf, 4, 16), (bf, 8, 16), (f32, 16), (f32, 4)
    pos, offs, w, dc, gu = (i32, 4, 2), (i32, 4), (bf, 3, 32, 16), (bf, 8, 32), (bf, 8, 32)
    return [
        (moe.moe_dispatch, dict(x=x, topk_ids=pos), dict(num_experts=3)),
        (moe.moe_dispatch_backward, dict(drows=rows, pos=pos), {}),
        (moe.moe_combine, dict(y=rows, pos=pos, weights=(f32, 4, 2)), {}),
        (moe.moe_combine_backward, dict(dout=x, y=rows, pos=pos, pair_ids=(i32, 8), weights=(f32, 4, 2)), {}),
        (moe.moe_pre_norm, dict(x=x, weight=vec), {}),
        (moe.moe_pre_norm_backward, dict(dh=x, x=x, weight=vec, rstd=t, dresidual=x), {}),
        (moe.moe_post_norm, dict(y=x, residual=x, weight=vec, gate=(bf, 4), next_weight=vec), dict(gate_kind="token")),
        (moe.moe_post_norm_backward, dict(dout=x, y=x, weight=vec, rstd=t, gate=x), dict(gate_kind="full")),
        (moe.moe_expert_gemm, dict(a=rows, w=w, expert_offsets=offs), {}),
        (moe.moe_expert_gemm_silu_mul, dict(a=rows, w=w, expert_offsets=offs), {}),
        (moe.moe_expert_gemm_dgrad, dict(dc=dc, w=(bf, 3, 32, 16), expert_offsets=offs, gate_up=gu), {}),
        (moe.moe_expert_gemm_wgrad, dict(dc=dc, a=rows, expert_offsets=offs), {}),
    ]


class Launched(Exception):
    pass


@pytest.fixture
def no_launch(monkeypatch):
    """Device 0 is current; a call that gets as far as its results' memory stops there."""
    def stop(*_):
        raise Launched
    monkeypatch.setattr(ops, "_device", lambda: 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(ops, "_empty_strided", stop)


@pytest.mark.parametrize("f,operands,other", device_calls(), ids=lambda v: getattr(v, "__name__", ""))
def test_operands_on_another_device_are_refused(f, operands, other, no_launch):
    make = lambda bad=None: {k: OnDevice(*v, device=int(k == bad)) for k, v in operands.items()}  # noqa: E731
    with pytest.raises(Launched):
        f(**make(), **other)
    for name in operands:
        with pytest.raises(ValueError, match=f"{name}.* is on cuda:1, but the current device is cuda:0"):
            f(**make(name), **other)


def test_gradients_on_another_device_are_refused(no_launch):
    at = lambda d: OnDevice(torch.float32, 5, device=d)  # noqa: E731
    with pytest.raises(Launched):
        moe.moe_clip_grads([at(0), at(0)], 1.0, out=[at(0), at(0)])
    with pytest.raises(ValueError, match=r"grads\[1\] is on cuda:1"):
        moe.moe_clip_grads([at(0), at(1)], 1.0)
    with pytest.raises(ValueError, match=r"grads\[0\] is on cuda:1"):
        moe.moe_clip_grads([at(1), at(1)], 1.0)
    with pytest.raises(ValueError, match=r"out\[1\] .* on its device"):
        moe.moe_clip_grads([at(0), at(0)], 1.0, out=[at(0), at(1)])


def test_layer_operands_on_another_device_are_refused(no_launch):
    y, pos = (torch.float32, 8, 16), (torch.int32, 8)
    out = OnDevice(torch.bfloat16, 4, 16)
    for bad in "y", "pos":
        with pytest.raises(ValueError, match=f"{bad} is on cuda:1"):
            moe.moe_unpermute_sum(OnDevice(*y, device=int(bad == "y")), OnDevice(*pos, device=int(bad == "pos")), 4, 2, out)


def test_binding_without_torchs_private_functions(monkeypatch):
    """Where torch lacks the quick forms, the public ones stand in."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location(ops.__name__ + "_public", ops.__file__)
    public = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, public)
    spec.loader.exec_module(public)

    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream)
    assert public._device is torch.cuda.current_device and public._raw_stream(0) == 77


@pytest.mark.parametrize("change,code", [
    (dict(grads=(0x10000, 0x10000)), INVALID),                                 # a tensor given twice, in place
    (dict(grads=(0x10000, 0x10004), dtype=(0, 0)), INVALID),                   # its second half beside it
    (dict(grads=(0x10004, 0x10000), dtype=(0, 0), numel=(9, 3)), INVALID),
    (dict(out=(0x20000, 0x10000)), INVALID),                                   # results in each other's gradients
    (dict(out=(0x30000, 0x30000)), INVALID),
    (dict(out=(0x10004, 0x40000)), INVALID),                                   # a result in its own, moved
    (dict(grads=(0x10000, 0x10000), out=(0x10000, 0x30000), dtype=(0, 0)), INVALID),   # read and written in place
    (dict(grads=(0x10000, 0x10000), out=(0x30000, 0x40000)), WORKSPACE),       # the same gradient read twice
    (dict(grads=(0x10000, 0x10008), dtype=(0, 0)), WORKSPACE),                 # neighbours
    (dict(grads=(0x10000, 0x10000), numel=(4, 0)), WORKSPACE),                 # nothing in the second
])
def test_clip_refuses_results_that_overlap(change, code):
    assert clip(wsb=0, **change) == code


def test_clip_refuses_overlaps_among_many():
    n = 1000
    for at, code in ((0x10000 + 64 * 500, INVALID), (0x10000 + 64 * n, WORKSPACE)):
        g = (ctypes.c_void_p * n)(*[0x10000 + 64 * ((i * 7) % n) for i in range(n - 1)], at)
        args = ((ctypes.c_int64 * n)(*[16] * n), (ctypes.c_int32 * n)(*[2] * n), n, 0, 1.0, 1e-6, P, P, 0, None)
        assert ops.lib().moe_clip_grads(g, g, *args) == code


@pytest.mark.parametrize("f,operands,other", [
    (moe.moe_dispatch, dict(x=(torch.bfloat16, 2 ** 32 + 4, 8), topk_ids=(torch.int32, 2 ** 32 + 4, 2)), dict(num_experts=3)),
    (moe.moe_dispatch, dict(x=(torch.bfloat16, 4, 2 ** 32 + 8), topk_ids=(torch.int32, 4, 2)), dict(num_experts=3)),
    (moe.moe_dispatch, dict(x=(torch.bfloat16, 4, 8), topk_ids=(torch.int32, 4, 2 ** 32 + 2)), dict(num_experts=3)),
    (moe.moe_dispatch, dict(x=(torch.bfloat16, 4, 8), topk_ids=(torch.int32, 4, 2)), dict(num_experts=2 ** 32 + 3)),
    (moe.moe_dispatch, dict(x=(torch.bfloat16, 4, 8), topk_ids=(torch.int32, 4, 2)), dict(num_experts=3 - 2 ** 32)),
    (moe.moe_dispatch_backward, dict(drows=(torch.bfloat16, 8, 8), pos=(torch.int32, 2 ** 32 + 4, 2)), {}),
    (moe.moe_combine, dict(y=(torch.bfloat16, 8, 8), pos=(torch.int32, 4, 2 ** 32 + 2)), {}),
    (moe.moe_pre_norm, dict(x=(torch.bfloat16, 2 ** 32 + 4, 8), weight=(torch.float32, 8)), {}),
    (moe.moe_post_norm, dict(y=(torch.bfloat16, 2 ** 32 + 4, 8), residual=(torch.bfloat16, 2 ** 32 + 4, 8),
                             weight=(torch.float32, 8)), {}),
    (moe.moe_expert_gemm, dict(a=(torch.bfloat16, 8, 16), w=(torch.bfloat16, 3, 2 ** 32 + 8, 16),
                               expert_offsets=(torch.int32, 4)), {}),
    (moe.moe_expert_gemm_dgrad, dict(dc=(torch.bfloat16, 8, 16), w=(torch.bfloat16, 3, 16, 2 ** 32 + 8),
                                     expert_offsets=(torch.int32, 4)), {}),
], ids=lambda v: getattr(v, "__name__", ""))
def test_sizes_past_32_bits_are_refused(f, operands, other, no_launch):
    """The C ABI takes int sizes, to which ctypes cuts silently."""
    with pytest.raises(ValueError, match=r"2\^31"):
        f(**{k: OnDevice(*v) for k, v in operands.items()}, **other)


@pytest.mark.parametrize("f,operands,other", device_calls(), ids=lambda v: getattr(v, "__name__", ""))
def test_operands_that_autograd_follows_draw_a_warning(f, operands, other, no_launch):
    """The results have no grad_fn, so backward() would pass these operands by in silence."""
    for name, (dtype, *_) in operands.items():
        if not dtype.is_floating_point:
            continue
        made = {k: OnDevice(*v) for k, v in operands.items()}
        made[name].requires_grad = True
        with pytest.warns(UserWarning, match=f"^{f.__name__} records nothing for autograd") as seen, pytest.raises(Launched):
            f(**made, **other)
        assert len(seen) == 1 and seen[0].filename == __file__
        with warnings.catch_warnings(), torch.no_grad(), pytest.raises(Launched):
            warnings.simplefilter("error")
            f(**made, **other)
    with warnings.catch_warnings(), pytest.raises(Launched):
        warnings.simplefilter("error")
        f(**{k: OnDevice(*v) for k, v in operands.items()}, **other)


@pytest.mark.parametrize("T,topk,E", [(152 * 65536, 65536, 8), (2 ** 31 - 1, 2 ** 31 - 1, 8), (16384, 2 ** 30, 8),
                                      (2 ** 30, 2, 8), (300000, 33, 8), (300000, 2, 1025)])
def test_dispatch_workspace_size_of_refused_sizes(T, topk, E):
    """The chunks of so many pairs have no int size: it must not divide by what is left of one."""
    assert ops.lib().moe_dispatch_workspace_size(T, topk, E) == 0
    assert dispatch(T=T, topk=topk, E=E) == SHAPE
