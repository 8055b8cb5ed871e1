"""Training steps of one mixture-of-experts block on the package's training operators.

The block: RMS norm -> router -> token rows sorted by expert -> w13 with SiLU(gate)*up -> w2 -> the
router-weighted sum back to the tokens -> RMS norm with a learned gate per channel, scaled and added
to the residual.  Its gradient runs the operators' backward passes in reverse; the gradients are
clipped by their global norm and applied by plain gradient descent.  The router's logits (one
small product) and the gradient of its softmax over the chosen experts are plain torch.

    python examples/train_moe_block.py --tokens 4096 --hidden 2048 --inter 768 --experts 128 --topk 8 --steps 20
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_fp8_mixture_topk_gb300 as moe  # noqa: E402

BLOCK_SCALE = 0.5


def init_params(H, I, E, seed=0, device="cuda"):
    """Weights of the block: experts in bf16, the small ones in fp32 (the channel gate in the rows' type)."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, std: torch.randn(*s, generator=g) * std  # noqa: E731
    p = {"pre": 1 + rn(H, std=0.1), "router": rn(E, H, std=H ** -0.5), "w13": rn(E, 2 * I, H, std=H ** -0.5).bfloat16(),
         "w2": rn(E, H, I, std=I ** -0.5).bfloat16(), "post": 1 + rn(H, std=0.1), "gate": (1 + rn(H, std=0.1)).bfloat16()}
    return {k: v.to(device) for k, v in p.items()}


def forward(p, x, topk):
    """out [T, H] and what the gradient needs."""
    E = p["router"].shape[0]
    h, r_pre = moe.moe_pre_norm(x, p["pre"])
    logits = h.float() @ p["router"].T
    ids, weights = moe.moe_route_topk(logits, topk)
    d = moe.moe_dispatch(h, ids, E)
    act, gate_up = moe.moe_expert_gemm_silu_mul(d.rows, p["w13"], d.expert_offsets)
    y = moe.moe_expert_gemm(act, p["w2"], d.expert_offsets)
    z = moe.moe_combine(y, d.pos, weights)
    post = moe.moe_post_norm(z, x, p["post"], gate=p["gate"], gate_kind="channel", block_scale=BLOCK_SCALE)
    return post.out, dict(x=x, h=h, r_pre=r_pre, ids=ids, weights=weights, d=d, act=act, gate_up=gate_up, y=y, z=z,
                          r_post=post.rstd)


def backward(p, s, dout):
    """Gradients of the parameters and of x for the gradient of out."""
    d, off, g = s["d"], s["d"].expert_offsets, {}
    post = moe.moe_post_norm_backward(dout, s["z"], p["post"], s["r_post"], gate=p["gate"], gate_kind="channel",
                                      block_scale=BLOCK_SCALE)
    g["post"], g["gate"] = post.dweight, post.dgate
    dy, dweights = moe.moe_combine_backward(post.dy, s["y"], d.pos, d.pair_ids, s["weights"])
    g["w2"] = moe.moe_expert_gemm_wgrad(dy, s["act"], off)
    dgate_up = moe.moe_expert_gemm_dgrad(dy, p["w2"], off, gate_up=s["gate_up"])
    g["w13"] = moe.moe_expert_gemm_wgrad(dgate_up, d.rows, off)
    dh = moe.moe_dispatch_backward(moe.moe_expert_gemm_dgrad(dgate_up, p["w13"], off), d.pos)
    # the router: its weights are a softmax over the chosen logits
    w = s["weights"]
    chosen = w * (dweights - (w * dweights).sum(1, keepdim=True))
    dlogits = torch.zeros(w.shape[0], p["router"].shape[0], device=w.device).scatter_(1, s["ids"].long(), chosen)
    g["router"] = dlogits.T @ s["h"].float()
    dh = (dh.float() + dlogits @ p["router"]).to(dh.dtype)
    g["x"], g["pre"] = moe.moe_pre_norm_backward(dh, s["x"], p["pre"], s["r_pre"], dresidual=post.dresidual)
    return g


def train_step(p, x, target, topk, lr, max_norm=1.0):
    """One step towards `target` (mean squared error); the parameters change in place.  Returns (loss,
    the gradients' norm before clipping), on the device."""
    out, saved = forward(p, x, topk)
    diff = out.float() - target
    grads = backward(p, saved, (diff * (2.0 / diff.numel())).to(out.dtype))
    names = sorted(p)
    norm = moe.moe_clip_grads([grads[n] for n in names], max_norm)
    for n in names:
        p[n].add_(grads[n].to(p[n].dtype), alpha=-lr)
    return diff.square().mean(), norm


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inter", 768), ("experts", 128), ("topk", 8), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args(argv)
    p = init_params(a.hidden, a.inter, a.experts)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g).bfloat16().cuda()
    target = x.float() + 0.5 * torch.randn(a.hidden, a.hidden, generator=g).cuda().mul_(a.hidden ** -0.5).T.matmul(x.float().T).T
    losses = []
    for step in range(a.steps):
        loss, norm = train_step(p, x, target, a.topk, a.lr)
        losses.append(loss.item())
        print(f"step {step}: loss {losses[-1]:.5f}, gradient norm {norm.item():.4f}")
    return losses


if __name__ == "__main__":
    main()
