"""A mixture-of-experts block of trained 16-bit weights, served in 4 bits.

The experts' weights go into MXFP4 or NVFP4 once, at load time; a step then runs router -> token rows sorted by expert -> rows in
4 bits -> first product with SiLU(gate)*up and its result in 4 bits -> second product -> router-weighted sum, and is captured
in a graph.  Prints the steps' time and how far 4 bits take the result from the 16-bit block's.

    python examples/serve_fp4_block.py --tokens 4096 --hidden 2048 --inter 768 --experts 128 --topk 8 --format mxfp4
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_fp8_mixture_topk_gb300 as moe  # noqa: E402


def load(p, fmt):
    """The 4-bit experts of 16-bit weights w13 [E, 2I, H], w2 [E, H, I]: codes, packed scales, expert scales (nvfp4)."""
    q = {"router": p["router"], "format": fmt}
    for name, gate_up in (("w13", True), ("w2", False)):
        if fmt == "mxfp4":
            codes, scales = moe.moe_mxfp4_quant_weight(p[name])
            total = None
        else:
            codes, scales, total = moe.moe_nvfp4_quant_weight(p[name])
        q[name] = (codes, moe.moe_fp4_pack_scales(scales, fmt, gate_up=gate_up), total)
    return q


def forward(q, x, topk):
    """The block of x [T, H] (bf16) on 4-bit experts."""
    E = q["router"].shape[0]
    route = moe.moe_router(x.float() @ q["router"].T, topk)
    d = moe.moe_dispatch(x, route.ids, E)
    rows = moe.moe_fp4_quant(d.rows, q["format"], d.expert_offsets)
    act = moe.moe_fp4_expert_gemm_silu_mul_quant(rows, *q["w13"])
    return moe.moe_combine(moe.moe_fp4_expert_gemm(act, *q["w2"]), d.pos, route.weights)


def forward_16(p, x, topk):
    """The same on the 16-bit experts."""
    route = moe.moe_router(x.float() @ p["router"].T, topk)
    d = moe.moe_dispatch(x, route.ids, p["router"].shape[0])
    act, _ = moe.moe_expert_gemm_silu_mul(d.rows, p["w13"], d.expert_offsets, save_gate_up=False)
    return moe.moe_combine(moe.moe_expert_gemm(act, p["w2"], d.expert_offsets), d.pos, route.weights)


def weights(H, I, E, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, std: (torch.randn(*s, generator=g) * std).cuda()  # noqa: E731
    return {"router": rn(E, H, std=H ** -0.5), "w13": rn(E, 2 * I, H, std=H ** -0.5).bfloat16(),
            "w2": rn(E, H, I, std=I ** -0.5).bfloat16()}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inter", 768), ("experts", 128), ("topk", 8), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--format", choices=["mxfp4", "nvfp4"], default="mxfp4")
    a = ap.parse_args(argv)
    p = weights(a.hidden, a.inter, a.experts)
    q = load(p, a.format)
    x = torch.randn(a.tokens, a.hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward(q, x, a.topk)                    # the first step sets up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(q, x, a.topk)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    want = forward_16(p, x, a.topk).float()
    off = ((out.float() - want).norm() / want.norm()).item()
    print(f"{a.format}: {start.elapsed_time(end) / a.steps * 1000:.1f} us a step, {off:.4f} from 16 bits")
    return off


if __name__ == "__main__":
    main()
