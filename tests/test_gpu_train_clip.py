"""Global gradient norm and clipping against 64-bit values."""
import math

import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from train_testutil import DTYPES, check, gen, ids_of, offset_copy, rand

pytestmark = pytest.mark.gpu

# squares are summed in fp32 over at most 32 elements of a thread's share (fp64 beyond; 128 elements
# where a tensor's address allows no vectors), the root halves that; then one rounding to fp32, and
# for the clipped values the scale's rounding
NORM = 128 / 2 + 1


def norm64(grads, kind):
    if kind == 2:
        return math.sqrt(sum((t.double() ** 2).sum().item() for t in grads))
    return max([t.double().abs().max().item() for t in grads if t.numel()], default=0.0)


@pytest.mark.parametrize("norm_type", [2, float("inf")])
@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("dtype", DTYPES + ["mixed"], ids=lambda d: d if d == "mixed" else ids_of(d))
@pytest.mark.parametrize("sizes", [[1], [7, 0, 33], [16384, 16385, 3], [100000, 1, 65536, 0, 131071], [40] * 33,
                                   [5] * 129, [9] * 1000], ids=lambda s: f"{len(s)}x{s[0]}")
def test_clip(sizes, dtype, inplace, norm_type):
    g = gen(len(sizes))
    kinds = [DTYPES[i % 3] if dtype == "mixed" else dtype for i in range(len(sizes))]
    grads = [rand(g, n, dtype=t, std=0.1) for n, t in zip(sizes, kinds)]
    before = [t.clone() for t in grads]
    total = norm64(grads, norm_type)
    for limit in (total / 3, total * 2):
        for t, b in zip(grads, before):
            t.copy_(b)
        out = None if inplace else [torch.full_like(t, 7.0) for t in grads]
        got = moe.moe_clip_grads(grads, limit, norm_type=norm_type, out=out)
        assert got.dtype == torch.float32 and got.dim() == 0
        check(got, torch.tensor(total, dtype=torch.float64), roundings=NORM, name="norm")
        scale = min(1.0, limit / (total + 1e-6))
        for t, b in zip(grads if inplace else out, before):
            if scale == 1.0:
                assert torch.equal(t, b)
            else:
                check(t, b.double() * scale, roundings=NORM + 4, name="clipped")
        if not inplace:
            assert all(torch.equal(t, b) for t, b in zip(grads, before))


def test_views_at_odd_addresses():
    g = gen(2)
    grads = [offset_copy(rand(g, n, dtype=t), by) for n in (1, 31, 70001) for by in (1, 3) for t in DTYPES]
    before = [t.clone() for t in grads]
    total = norm64(grads, 2)
    got = moe.moe_clip_grads(grads, 1.0)
    check(got, torch.tensor(total, dtype=torch.float64), roundings=NORM, name="norm")
    for t, b in zip(grads, before):
        check(t, b.double() / (total + 1e-6), roundings=NORM + 4, name="clipped")


def test_magnitudes_whose_squares_leave_fp32():
    for dtype in (torch.float32, torch.bfloat16):
        for size in (1e-25, 1e-22, 3e-19, 1e19, 1e25, 1e30):
            t = torch.full((5000,), size, device="cuda", dtype=dtype)
            t[::3] = 0
            total = norm64([t], 2)
            got = moe.moe_clip_grads([t.clone()], float("inf"))
            check(got, torch.tensor(total, dtype=torch.float64), roundings=NORM, name=f"{dtype} {size}")
    # a share of large values beside one of small values
    t = torch.cat([torch.full((40000,), 1e20, device="cuda"), torch.full((40000,), 1e-3, device="cuda")])
    check(moe.moe_clip_grads([t.clone()], 1.0), torch.tensor(norm64([t], 2), dtype=torch.float64), roundings=NORM,
          name="both")


def test_not_finite():
    for norm_type in (2, float("inf")):
        a, b = torch.ones(70000, device="cuda"), torch.ones(9, device="cuda", dtype=torch.bfloat16)
        a[69999] = float("inf")
        total = moe.moe_clip_grads([a, b], 1.0, norm_type=norm_type)
        assert math.isinf(total.item())
        assert torch.isnan(a[69999]) and torch.equal(a[:69999], torch.zeros(69999, device="cuda"))
        assert torch.equal(b, torch.zeros_like(b))
        b = torch.ones(9, device="cuda", dtype=torch.float16)
        b[4] = float("nan")
        a = torch.ones(70000, device="cuda")
        total = moe.moe_clip_grads([a, b], 1.0, norm_type=norm_type)
        assert math.isnan(total.item()) and torch.isnan(a).all() and torch.isnan(b).all()


def test_nothing_and_zeros():
    assert moe.moe_clip_grads([], 1.0).item() == 0
    assert moe.moe_clip_grads([torch.zeros(0, device="cuda")], 1.0).item() == 0
    z = torch.zeros(100, device="cuda")
    assert moe.moe_clip_grads([z], 1.0).item() == 0 and torch.equal(z, torch.zeros(100, device="cuda"))
    o = torch.ones(100, device="cuda")
    assert abs(moe.moe_clip_grads([o], 0.0).item() - 10) < 1e-5 and torch.equal(o, torch.zeros(100, device="cuda"))


def test_more_tensors_than_a_launch_takes():
    g = gen(8)
    grads = [rand(g, 1 + i % 37, dtype=DTYPES[i % 3]) for i in range(2500)]
    before = [t.clone() for t in grads]
    total = norm64(grads, 2)
    check(moe.moe_clip_grads(grads, 2.0), torch.tensor(total, dtype=torch.float64), roundings=NORM, name="norm")
    for t, b in zip(grads, before):
        check(t, b.double() * (2.0 / (total + 1e-6)), roundings=NORM + 4, name="clipped")


def test_large_tensor_repeats_and_graph():
    """More chunks than CTAs; the same bits every time; a graph replayed on new values."""
    g = torch.Generator(device="cuda").manual_seed(4)
    t = torch.randn(90_000_001, generator=g, device="cuda", dtype=torch.bfloat16)
    small = torch.randn(1001, generator=g, device="cuda")
    total = norm64([t, small], 2)
    outs = [[torch.empty_like(t), torch.empty_like(small)] for _ in range(2)]
    a = moe.moe_clip_grads([t, small], 5.0, out=outs[0])
    b = moe.moe_clip_grads([t, small], 5.0, out=outs[1])
    check(a, torch.tensor(total, dtype=torch.float64), roundings=NORM, name="norm")
    assert torch.equal(a, b) and torch.equal(outs[0][0], outs[1][0])
    want = t.double() * (5.0 / (total + 1e-6))
    assert ((outs[0][0].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -16) * want.abs() + 1e-38).all()
    del want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = moe.moe_clip_grads([t, small], 5.0, out=outs[0])
    t.normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    check(n, torch.tensor(norm64([t, small], 2), dtype=torch.float64), roundings=NORM, name="norm of the replay")
    again = moe.moe_clip_grads([t, small], 5.0, out=outs[1])
    assert torch.equal(n, again) and torch.equal(outs[0][0], outs[1][0])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("src,dst", [(0, 1), (1, 0), (3, 2), (5, 5), (7, 4)])
def test_results_elsewhere_between_boundaries(src, dst, dtype):
    """Gradients and results at addresses of their own; nothing beside the results is written."""
    g = gen(src * 8 + dst)
    sizes = [1, 2, 7, 8, 9, 31, 1023, 4093, 4096, 4099, 8200, 70001]
    grads = [offset_copy(rand(g, n, dtype=dtype), src) for n in sizes]
    around = [torch.full((n + dst + 9,), 5.0, dtype=dtype, device="cuda") for n in sizes]
    out = [b[dst:dst + n] for b, n in zip(around, sizes)]
    total = norm64(grads, 2)
    got = moe.moe_clip_grads(grads, total / 2, out=out)
    check(got, torch.tensor(total, dtype=torch.float64), roundings=NORM, name="norm")
    for t, o, b, n in zip(grads, out, around, sizes):
        check(o, t.double() * (total / 2 / (total + 1e-6)), roundings=NORM + 4, name="clipped")
        assert (b[:dst] == 5).all() and (b[dst + n:] == 5).all()


def test_autograd_sees_that_the_results_changed():
    """What autograd saved of a clipped tensor is no longer what it saved: backward() refuses, as after torch's own
    in-place operations, in place of a wrong gradient."""
    other = torch.ones(7, device="cuda")
    for out in (None, "out"):
        w = torch.ones(7, device="cuda", requires_grad=True)
        saved = w.exp()
        grads = [other.clone(), saved.detach()] if out is None else [other.clone(), other.clone()]
        before = [g._version for g in grads]
        moe.moe_clip_grads(grads, 0.5, out=None if out is None else [torch.empty_like(other), saved.detach()])
        assert [g._version > b for g, b in zip(grads, before)] == [out is None] * 2
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()
    with torch.inference_mode():
        g = torch.ones(7, device="cuda")
    assert moe.moe_clip_grads([g], 1.0) > 1 and g[0] < 1
    assert moe.moe_clip_grads([], 1.0) == 0


def test_a_tensor_past_two_to_the_31_elements():
    g = torch.Generator(device="cuda").manual_seed(9)
    n = 2 ** 31 + 4099
    t = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    t[-9000:] = torch.randn(9000, generator=g, device="cuda").bfloat16()
    end = t[-9000:].double()
    total = math.sqrt(n - 9000 + end.square().sum().item())
    got = moe.moe_clip_grads([t], total / 4)
    check(got, torch.tensor(total, dtype=torch.float64), roundings=NORM, name="norm")
    check(t[-9000:], end * (total / 4 / (total + 1e-6)), roundings=NORM + 4, name="the end")
    assert (t[:-9000] == 0.25).all()
