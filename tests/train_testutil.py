"""Helpers of the training operators' tests: tolerances that count roundings, and odd layouts.

A result rounded once to type t is off by at most half a step, finfo(t).eps / 2 of its size (below t's normal
range: half its smallest number).  A sum of n terms in fp32 is off by at most n * 2^-24 of the sum of
the terms' magnitudes, whatever its order."""
import torch

import block_fp8_mixture_topk_gb300 as moe

U32 = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
ids_of = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}.get


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, size=None, roundings=0.0, name=""):
    """|got - ref| <= half a step of got's type at ref, plus `roundings` fp32 half-steps of `size` (the
    sum of the magnitudes that went into each value), shifted into the rounded value."""
    ref = ref.double().cpu()
    g = got.detach().double().cpu()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    before = roundings * U32 * (size.double().cpu() if size is not None else ref.abs())
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    tol = half_step(got.dtype) * (ref.abs() + before) + before + tiny
    same_nan = torch.equal(torch.isnan(g), torch.isnan(ref))
    assert same_nan, f"{name}: NaN in other places"
    fine = torch.isfinite(ref)
    assert torch.equal(g[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{name}: infinities differ"
    bad = (g - ref).abs()[fine] > tol[fine]
    worst = ((g - ref).abs()[fine] / tol[fine]).max().item() if fine.any() else 0.0
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {worst:.2f} of the tolerance"


def rand(g, *shape, dtype=torch.float32, std=1.0, device="cuda"):
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(device)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def offset_copy(t, by=1):
    """The same values at an address `by` elements past an allocation's start (rows dense)."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


def strided_copy(t, pad, lead=0):
    """The same rows inside a wider matrix (columns lead .. lead + cols of cols + pad)."""
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    big[:, lead:lead + t.shape[1]] = t
    return big[:, lead:lead + t.shape[1]]


def status_clear():
    moe.moe_get_device_status(clear=True)


def status():
    return moe.moe_get_device_status(clear=True)
