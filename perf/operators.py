"""The operators that train a mixture-of-experts block around its experts, case by case, in plain torch.

Four operators, each with its gradient:

  tokens   token rows sorted by expert and back: the stable sort of the routed pairs, the gather of
           the rows, the router-weighted sum that brings the experts' rows back to the tokens, and
           the gradients of both;
  norms    the RMS norm before the block, and the norm after it fused with the block's gate, the
           scaled residual and the next block's norm, and the gradients of both;
  experts  the experts' products over rows sorted by expert (SiLU(gate)*up fused into the first),
           the gradient of their rows and the gradient of their weights;
  clip     the global norm of many gradient tensors, and their clipping.

Where `own` is false, run() computes them in elementary torch operations, in 32 bits; where it is true,
through the package's entry points.  exact() is the same in 64 bits from the definitions.

Shapes are those of the package's workloads (DeepSeek-V3-, Qwen3-30B-A3B- and Mixtral-shaped layers).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


def _moe():
    import block_fp8_mixture_topk_gb300 as moe
    return moe


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of eight requests: latency
        {"name": "tokens_decode", "op": "tokens", "dir": "forward", "T": 8, "H": 7168, "E": 256, "k": 8,
         "dtype": "bf16", "skew": 0.0, "drop": 0.0},
        # a DeepSeek-V3-shaped prefill or training micro-batch
        {"name": "tokens_dsv3", "op": "tokens", "dir": "forward", "T": 4096, "H": 7168, "E": 256, "k": 8,
         "dtype": "bf16", "skew": 0.0, "drop": 0.0},
        # the backward pass of a long batch whose router is skewed, some pairs dropped by a capacity limit
        {"name": "tokens_qwen3_backward", "op": "tokens", "dir": "backward", "T": 16384, "H": 2048, "E": 128, "k": 8,
         "dtype": "bf16", "skew": 1.2, "drop": 0.02},
        # one token through the norms of a block whose output has a per-token gate: latency
        {"name": "norms_decode", "op": "norms", "dir": "forward", "T": 1, "H": 7168, "dtype": "bf16",
         "weight": "fp32", "gate": "token", "sigmoid": True, "next": True},
        # a prefill's rows with a learned scale per channel on the block
        {"name": "norms_dsv3", "op": "norms", "dir": "forward", "T": 4096, "H": 7168, "dtype": "bf16",
         "weight": "bf16", "gate": "channel", "sigmoid": False, "next": True},
        # a ragged training batch with a gate for every element, and its gradient
        {"name": "norms_odd_backward", "op": "norms", "dir": "backward", "T": 5003, "H": 2880, "dtype": "bf16",
         "weight": "fp32", "gate": "full", "sigmoid": True, "next": False},
        # the gradients of a tiny layer: latency
        {"name": "clip_tiny", "op": "clip", "layers": 1, "H": 256, "I": 256, "E": 4, "grads": "fp32", "norm": "2",
         "over": 3.7},
        # the gradients of one Qwen3-30B-A3B-shaped layer
        {"name": "clip_qwen3", "op": "clip", "layers": 1, "H": 2048, "I": 768, "E": 128, "grads": "bf16", "norm": "2",
         "over": 3.7},
        # the first product of eight decoding requests: few rows, every touched expert's weights read once
        {"name": "experts_decode", "op": "experts", "dir": "forward", "T": 8, "k": 8, "E": 128, "K": 2048, "N": 1536,
         "dtype": "bf16", "silu": True, "skew": 0.0, "drop": 0.0},
        # the first product of a long skewed batch
        {"name": "experts_qwen3", "op": "experts", "dir": "forward", "T": 16384, "k": 8, "E": 128, "K": 2048,
         "N": 1536, "dtype": "bf16", "silu": True, "skew": 1.2, "drop": 0.0},
        # the rows' gradient through the second product and SiLU(gate)*up, few large experts
        {"name": "experts_mixtral_rows", "op": "experts", "dir": "rows", "T": 512, "k": 2, "E": 8, "K": 14336,
         "N": 4096, "dtype": "fp16", "silu": True, "skew": 0.0, "drop": 0.0},
        # the weights' gradient of the long skewed batch
        {"name": "experts_qwen3_weights", "op": "experts", "dir": "weights", "T": 16384, "k": 8, "E": 128, "K": 2048,
         "N": 1536, "dtype": "bf16", "silu": False, "skew": 1.2, "drop": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "norms", "experts", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "tokens":
        k = rng.choice([1, 2, 4, 6, 8])
        T = _log(rng, 1, 16384)
        H = min(_log(rng, 64, 8192), max(64, (1 << 29) // (T * k * SIZES[dtype])))
        if rng.random() < 0.7:
            H = max(8, H // 8 * 8)
        return {"op": op, "dir": rng.choice(["forward", "backward"]), "T": T, "H": H, "E": _log(rng, max(8, k), 512),
                "k": k, "dtype": dtype, "skew": rng.choice([0.0, 1.2]), "drop": rng.choice([0.0, 0.05])}
    if op == "norms":
        T = _log(rng, 1, 16384)
        H = min(_log(rng, 64, 16384), max(64, (1 << 26) // (T * SIZES[dtype])))
        if rng.random() < 0.7:
            H = max(8, H // 8 * 8)
        return {"op": op, "dir": rng.choice(["forward", "backward"]), "T": T, "H": H, "dtype": dtype,
                "weight": rng.choice(["fp32", dtype]), "gate": rng.choice(["none", "token", "channel", "full"]),
                "sigmoid": rng.random() < 0.5, "next": rng.random() < 0.5}
    if op == "experts":
        k = rng.choice([1, 2, 4, 8])
        E = _log(rng, max(4, k), 256)
        K = _log(rng, 64, 8192) // 8 * 8
        N = min(_log(rng, 64, 8192), max(64, (1 << 29) // (E * K))) // 16 * 16
        T = _log(rng, 1, 16384)
        T = max(1, min(T, int(3e11 / (k * K * N)), (1 << 28) // (k * max(K, N))))
        direction = rng.choice(["forward", "rows", "weights"])
        return {"op": op, "dir": direction, "T": T, "k": k, "E": E, "K": K, "N": N,
                "dtype": rng.choice(["bf16", "fp16"]), "silu": direction != "weights" and rng.random() < 0.5,
                "skew": rng.choice([0.0, 1.2]), "drop": rng.choice([0.0, 0.05])}
    return {"op": op, "layers": rng.randint(1, 8), "H": _log(rng, 65, 2048), "I": _log(rng, 33, 768),
            "E": _log(rng, 1, 8), "grads": rng.choice(["bf16", "fp16", "fp32", "mixed"]),
            "norm": rng.choice(["2", "2", "inf"]), "over": rng.choice([0.5, 3.7])}


def work(case):
    c, op = case, case["op"]
    if op == "tokens":
        b, T, P, H = SIZES[c["dtype"]], c["T"], c["T"] * c["k"], c["H"]
        if c["dir"] == "forward":   # x, y, ids, weights in; rows, out, the sort's tables out
            return {"bytes": b * H * (2 * T + 2 * P) + 4 * (2 * P + 2 * P + c["E"] + 1), "flops": 2 * P * H}
        # dout, y, drows, weights, tables in; dy, dweights, dx out
        return {"bytes": b * H * (2 * T + 3 * P) + 4 * (3 * P + P), "flops": 5 * P * H}
    if op == "norms":
        b, T, H, w = SIZES[c["dtype"]], c["T"], c["H"], SIZES[c["weight"]]
        gate = b * {"none": 0, "token": T, "channel": H, "full": T * H}[c["gate"]]
        nx = 1 if c["next"] else 0
        if c["dir"] == "forward":   # x, y in; h, out (and the next h) out
            return {"bytes": b * T * H * (4 + nx) + gate + w * H * (2 + nx) + 4 * T * (2 + nx),
                    "flops": T * H * (11 + 4 * nx)}
        # dh, x, dout, y, the residual's gradient in; dx, dy, dresidual, dgate, two weight gradients out
        return {"bytes": b * T * H * 8 + 2 * gate + (w + 4) * H * 2 + 8 * T, "flops": T * H * 26}
    if op == "experts":
        P, K, N = c["T"] * c["k"], c["K"], c["N"]
        b = SIZES[c["dtype"]]
        touched = int(round(min(c["E"], P) if P >= 4 * c["E"] else c["E"] * (1 - (1 - 1 / c["E"]) ** P)))
        flops = 2 * P * K * N
        if c["dir"] == "forward":   # rows, touched weights in; the product (and SiLU(gate)*up) out
            return {"bytes": b * (P * K + touched * K * N + P * N + (P * N // 2 if c["silu"] else 0)), "flops": flops}
        if c["dir"] == "rows":      # dc, touched weights (, gate and up) in; the rows' gradient out
            return {"bytes": b * (P * N + touched * K * N + P * K * (4 if c["silu"] else 1)), "flops": flops}
        return {"bytes": b * (P * N + P * K + c["E"] * K * N), "flops": flops}
    n = sum(math.prod(s) * SIZES[t] for s, t in _shapes(c))
    return {"bytes": 2 * n, "flops": sum(3 * math.prod(s) for s, _ in _shapes(c))}


def _shapes(c):
    """(shape, type) of each gradient tensor of `layers` blocks: experts, router, norms."""
    H, I, E = c["H"], c["I"], c["E"]
    per = [(E, 2 * I, H), (E, H, I), (E, H), (H,), (H,)]
    kinds = ["bf16", "fp16", "fp32", "fp32", "fp32"] if c["grads"] == "mixed" else [c["grads"]] * 5
    return [(s, t) for _ in range(c["layers"]) for s, t in zip(per, kinds)]


# ----------------------------------------------------------------------------------------- inputs
def _route(g, T, E, k, skew, drop):
    """Expert ids [T, k] of a router with a popularity skew; -1 where a pair is dropped."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits -= skew * torch.log(torch.arange(1, E + 1, device="cuda"))
    top = logits.topk(k, dim=1)
    ids = top.indices.to(torch.int32)
    weights = torch.softmax(top.values, dim=1)
    if drop:
        gone = torch.rand(T, k, generator=g, device="cuda") < drop
        gone |= torch.rand(T, 1, generator=g, device="cuda") < drop / 4   # tokens that lose every expert
        ids = torch.where(gone, -1, ids)
    return ids.contiguous(), weights.contiguous()


def _sort(ids, E):
    """Pairs stably sorted by expert: (expert_offsets [E+1], pair_ids [T*k], pos [T, k]), -1 = none."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat >= 0, flat, E)
    order = torch.argsort(key, stable=True)
    at = key[order]
    offsets = torch.searchsorted(at, torch.arange(E + 1, device=ids.device))
    pair_ids = torch.where(at < E, order, -1)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=ids.device)
    pos = torch.where(flat >= 0, pos, -1)
    return offsets.int(), pair_ids.int(), pos.int().reshape(ids.shape)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, std=1.0, dtype=None: (  # noqa: E731
        torch.randn(*s, generator=g, device="cuda", dtype=dtype or DTYPES[c["dtype"]]).mul_(std))
    s = {"case": c}
    if c["op"] == "tokens":
        T, H, P = c["T"], c["H"], c["T"] * c["k"]
        s["ids"], s["weights"] = _route(g, T, c["E"], c["k"], c["skew"], c["drop"])
        s["y"] = rn(P, H)
        if c["dir"] == "forward":
            s["x"] = rn(T, H)
        else:
            s["offsets"], s["pair_ids"], s["pos"] = _sort(s["ids"], c["E"])
            s["dout"], s["drows"] = rn(T, H, std=0.1), rn(P, H, std=0.1)
    elif c["op"] == "norms":
        T, H = c["T"], c["H"]
        wt = DTYPES[c["weight"]]
        s["x"], s["y"] = rn(T, H), rn(T, H, std=0.3)
        s["w_pre"], s["w_post"], s["w_next"] = (rn(H, std=0.1, dtype=wt).add_(1) for _ in range(3))
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[c["gate"]]
        s["gate"] = rn(*shape) if shape else None
        s["residual_scale"], s["block_scale"] = 1.0, 0.22
        if c["dir"] == "backward":
            s["dh"], s["dout"] = rn(T, H, std=0.1), rn(T, H, std=0.1)
            s["rstd_pre"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["rstd_post"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS)
    elif c["op"] == "experts":
        K, N, E, P = c["K"], c["N"], c["E"], c["T"] * c["k"]
        ids, _ = _route(g, c["T"], E, c["k"], c["skew"], c["drop"])
        s["offsets"], _, _ = _sort(ids, E)
        s["ends"] = s["offsets"].tolist()
        if c["dir"] != "weights":
            s["w"] = rn(E, N, K, std=0.02)
        if c["dir"] != "rows":
            s["a"] = rn(P, K)
        if c["dir"] != "forward":
            s["dc"] = rn(P, N, std=0.1)
        if c["dir"] == "rows" and c["silu"]:
            s["gu"] = rn(P, 2 * K)
    else:
        shapes = _shapes(c)
        s["grads"] = [rn(*shape, std=1e-2 * (1 + i % 3), dtype=DTYPES[t]) for i, (shape, t) in enumerate(shapes)]
        # one buffer per type holds the clipped gradients
        s["flat"] = {t: torch.empty(sum(math.prod(x) for x, u in shapes if u == t), device="cuda", dtype=DTYPES[t])
                     for t in sorted({t for _, t in shapes})}
        at, s["out"] = dict.fromkeys(s["flat"], 0), []
        for shape, t in shapes:
            n = math.prod(shape)
            s["out"].append(s["flat"][t][at[t]:at[t] + n].view(shape))
            at[t] += n
        # a limit that the norm is `over` times (0.5: nothing to clip)
        size = [x.double().square().sum() for x in s["grads"]] if c["norm"] == "2" else [
            x.abs().max().double() for x in s["grads"]]
        total = torch.stack(size).sum().sqrt() if c["norm"] == "2" else torch.stack(size).max()
        s["max_norm"] = float(total) / c["over"]
    return s


# -------------------------------------------------------------------------------------- plain form
def _tokens(s):
    c = s["case"]
    T, k, H, dt = c["T"], c["k"], c["H"], DTYPES[c["dtype"]]
    if c["dir"] == "forward":
        offsets, pair_ids, pos = _sort(s["ids"], c["E"])
        rows = torch.where(pair_ids[:, None] >= 0, s["x"][pair_ids.clamp(min=0) // k], 0)
        w = torch.where(pos >= 0, s["weights"], 0.0)
        out = (s["y"][pos.clamp(min=0)].float() * w[:, :, None]).sum(1).to(dt)
        return {"rows": rows, "offsets": offsets, "pair_ids": pair_ids, "pos": pos, "out": out}
    pair_ids, pos = s["pair_ids"], s["pos"]
    real = pos >= 0
    pair = pair_ids.clamp(min=0)
    w = torch.where(pair_ids >= 0, s["weights"].reshape(-1)[pair], 0.0)
    dy = (s["dout"][pair // k].float() * w[:, None]).to(dt)
    at = pos.clamp(min=0)
    dw = (s["y"][at].float() * s["dout"].float()[:, None, :]).sum(2) * real
    dx = (s["drows"][at].float() * real[:, :, None]).sum(1).to(dt)
    return {"dy": dy, "dweights": dw, "dx": dx}


def _norm(x32, w):
    rstd = torch.rsqrt(x32.square().mean(1) + EPS)
    return x32 * rstd[:, None] * w.float(), rstd


def _gate(s):
    """The gate's value, broadcast over [T, H] (None: one)."""
    if s["gate"] is None:
        return None
    g = s["gate"].float()
    g = 1 / (1 + torch.exp(-g)) if s["case"]["sigmoid"] else g
    return g[:, None] if s["case"]["gate"] == "token" else g


def _norm_backward(dn, x32, w, rstd):
    """Gradients of x * rstd * w for the gradient dn of the result."""
    xh = x32 * rstd[:, None]
    t = dn * w.float()
    return rstd[:, None] * (t - xh * (t * xh).mean(1, keepdim=True)), (dn * xh).sum(0)


def _norms(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    x, y, g = s["x"].float(), s["y"].float(), _gate(s)
    if c["dir"] == "forward":
        h, rstd = _norm(x, s["w_pre"])
        z, rstd_post = _norm(y, s["w_post"])
        z = z if g is None else z * g
        out = (s["residual_scale"] * x + s["block_scale"] * z).to(dt)
        r = {"h": h.to(dt), "rstd": rstd, "out": out, "rstd_post": rstd_post}
        if c["next"]:   # the next block reads the stored stream
            nh, r["next_rstd"] = _norm(out.float(), s["w_next"])
            r["next_h"] = nh.to(dt)
        return r
    dout = s["dout"].float()
    dz = s["block_scale"] * dout
    dn = dz if g is None else dz * g
    dy, dw_post = _norm_backward(dn, y, s["w_post"], s["rstd_post"])
    r = {"dy": dy.to(dt), "dw_post": dw_post, "dresidual": (s["residual_scale"] * dout).to(dt)}
    if g is not None:
        dg = dz * (y * s["rstd_post"][:, None] * s["w_post"].float())
        dg = dg * (g * (1 - g)) if c["sigmoid"] else dg
        r["dgate"] = dg.sum(1).to(dt) if c["gate"] == "token" else dg.sum(0) if c["gate"] == "channel" else dg.to(dt)
    # the norm before the block: its input is also the residual, whose gradient joins here
    dx, r["dw_pre"] = _norm_backward(s["dh"].float(), x, s["w_pre"], s["rstd_pre"])
    r["dx"] = (dx + r["dresidual"].float()).to(dt)
    return r


def _experts(s):
    c = s["case"]
    K, N, E, P, dt = c["K"], c["N"], c["E"], c["T"] * c["k"], DTYPES[c["dtype"]]
    busy = [(e, s["ends"][e], s["ends"][e + 1]) for e in range(E) if s["ends"][e + 1] > s["ends"][e]]
    left = P - s["ends"][E]
    if c["dir"] == "weights":
        return {"dw": torch.stack([s["dc"][s["ends"][e]:s["ends"][e + 1]].float().T
                                   @ s["a"][s["ends"][e]:s["ends"][e + 1]].float() for e in range(E)]).to(dt)}
    if c["dir"] == "rows":
        da = torch.cat([s["dc"][lo:hi].float() @ s["w"][e].float() for e, lo, hi in busy]
                       + [torch.zeros(left, K, device="cuda")])
        if not c["silu"]:
            return {"da": da.to(dt)}
        gate, up = s["gu"][:, :K].float(), s["gu"][:, K:].float()
        sig = 1 / (1 + torch.exp(-gate))
        live = (torch.arange(P, device="cuda") < s["offsets"][E])[:, None]   # rows of no expert: zero
        return {"dgu": torch.where(live, torch.cat([da * up * sig * (1 + gate * (1 - sig)), da * gate * sig], 1),
                                   0.0).to(dt)}
    cc = torch.cat([s["a"][lo:hi].float() @ s["w"][e].float().T for e, lo, hi in busy]
                   + [torch.zeros(left, N, device="cuda")])
    if not c["silu"]:
        return {"c": cc.to(dt)}
    gate, up = cc[:, :N // 2], cc[:, N // 2:]
    return {"gu": cc.to(dt), "h": (gate / (1 + torch.exp(-gate)) * up).to(dt)}


def _clip(s):
    if s["case"]["norm"] == "2":
        total = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
    else:
        total = torch.stack([x.float().abs().max() for x in s["grads"]]).max()
    scale = torch.clamp(s["max_norm"] / (total + EPS), max=1.0)
    torch._foreach_copy_(s["out"], [(x.float() * scale).to(x.dtype) for x in s["grads"]])
    return {"total": total, **s["flat"]}


# ------------------------------------------------------------------------------------ entry points
def _own_tokens(s):
    moe, c = _moe(), s["case"]
    if c["dir"] == "forward":
        d = moe.moe_dispatch(s["x"], s["ids"], c["E"])
        out = moe.moe_combine(s["y"], d.pos, s["weights"])
        return {"rows": d.rows, "offsets": d.expert_offsets, "pair_ids": d.pair_ids, "pos": d.pos, "out": out}
    dy, dw = moe.moe_combine_backward(s["dout"], s["y"], s["pos"], s["pair_ids"], s["weights"])
    dx = moe.moe_dispatch_backward(s["drows"], s["pos"])
    return {"dy": dy, "dweights": dw, "dx": dx}


def _own_norms(s):
    moe, c = _moe(), s["case"]
    gate = dict(gate=s["gate"], gate_kind=c["gate"], gate_sigmoid=c["sigmoid"]) if s["gate"] is not None else {}
    scales = dict(residual_scale=s["residual_scale"], block_scale=s["block_scale"])
    if c["dir"] == "forward":
        h, rstd = moe.moe_pre_norm(s["x"], s["w_pre"], eps=EPS)
        p = moe.moe_post_norm(s["y"], s["x"], s["w_post"], eps=EPS, **gate, **scales,
                              next_weight=s["w_next"] if c["next"] else None)
        r = {"h": h, "rstd": rstd, "out": p.out, "rstd_post": p.rstd}
        if c["next"]:
            r["next_h"], r["next_rstd"] = p.next_h, p.next_rstd
        return r
    p = moe.moe_post_norm_backward(s["dout"], s["y"], s["w_post"], s["rstd_post"], **gate, **scales)
    dx, dw_pre = moe.moe_pre_norm_backward(s["dh"], s["x"], s["w_pre"], s["rstd_pre"], dresidual=p.dresidual)
    r = {"dy": p.dy, "dw_post": p.dweight, "dresidual": p.dresidual, "dx": dx, "dw_pre": dw_pre}
    if s["gate"] is not None:
        r["dgate"] = p.dgate
    return r


def _own_experts(s):
    moe, c = _moe(), s["case"]
    if c["dir"] == "weights":
        return {"dw": moe.moe_expert_gemm_wgrad(s["dc"], s["a"], s["offsets"])}
    if c["dir"] == "rows":
        if c["silu"]:
            return {"dgu": moe.moe_expert_gemm_dgrad(s["dc"], s["w"], s["offsets"], gate_up=s["gu"])}
        return {"da": moe.moe_expert_gemm_dgrad(s["dc"], s["w"], s["offsets"])}
    if c["silu"]:
        h, gu = moe.moe_expert_gemm_silu_mul(s["a"], s["w"], s["offsets"])
        return {"gu": gu, "h": h}
    return {"c": moe.moe_expert_gemm(s["a"], s["w"], s["offsets"])}


def _own_clip(s):
    total = _moe().moe_clip_grads(s["grads"], s["max_norm"], norm_type=float(s["case"]["norm"]), eps=EPS, out=s["out"])
    return {"total": total, **s["flat"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tokens": _own_tokens, "norms": _own_norms, "experts": _own_experts, "clip": _own_clip}[op](state)
    return {"tokens": _tokens, "norms": _norms, "experts": _experts, "clip": _clip}[op](state)


# ------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, r = s["case"], {}
    if c["op"] == "tokens":
        T, k, E, P = c["T"], c["k"], c["E"], c["T"] * c["k"]
        flat = s["ids"].reshape(-1)
        pairs = torch.cat([torch.nonzero(flat == e).reshape(-1) for e in range(E)])   # by expert, then by pair
        n = pairs.numel()
        place = torch.full((P,), -1, device="cuda")
        place[pairs] = torch.arange(n, device="cuda")
        y = torch.cat([s["y"], torch.zeros_like(s["y"][:1])])   # a dropped pair reads the zero row at -1
        if c["dir"] == "forward":
            rows = torch.zeros(P, c["H"], device="cuda", dtype=torch.float64)
            rows[:n] = s["x"][pairs // k].double()
            out = torch.zeros(T, c["H"], device="cuda", dtype=torch.float64)
            for j in range(k):
                out += s["weights"][:, j:j + 1].double() * y[place[j::k]].double()
            counts = torch.bincount(flat[flat >= 0].long(), minlength=E)
            full = torch.full((P,), -1, device="cuda")
            full[:n] = pairs
            return {"rows": rows, "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(),
                    "pair_ids": full.int(), "pos": place.int().reshape(T, k), "out": out}
        dr = torch.cat([s["drows"], torch.zeros_like(s["drows"][:1])])
        dy = torch.zeros(P, c["H"], device="cuda", dtype=torch.float64)
        dx = torch.zeros(T, c["H"], device="cuda", dtype=torch.float64)
        dw = torch.zeros(T, k, device="cuda", dtype=torch.float64)
        dout = s["dout"].double()
        for j in range(k):
            at = place[j::k]
            live = torch.nonzero(at >= 0).reshape(-1)
            dy[at[live]] = dout[live] * s["weights"][live, j:j + 1].double()
            dw[:, j] = torch.linalg.vecdot(dout, y[at].double())
            dx += dr[at].double()
        return {"dy": dy, "dweights": dw, "dx": dx}
    if c["op"] == "norms":
        dt, H = DTYPES[c["dtype"]], c["H"]
        x, y = s["x"].double(), s["y"].double()
        a, b = s["residual_scale"], s["block_scale"]
        g = torch.ones(1, 1, device="cuda", dtype=torch.float64) if s["gate"] is None else s["gate"].double()
        g = torch.sigmoid(g) if c["sigmoid"] and s["gate"] is not None else g
        g = g.reshape(-1, 1) if c["gate"] == "token" else g
        size = lambda v: torch.linalg.vecdot(v, v).div(H).add(EPS).sqrt()[:, None]  # noqa: E731
        if c["dir"] == "forward":
            out = a * x + b * g * (y / size(y) * s["w_post"].double())
            r = {"h": x / size(x) * s["w_pre"].double(), "rstd": 1 / size(x)[:, 0], "out": out,
                 "rstd_post": 1 / size(y)[:, 0]}
            if c["next"]:
                kept = out.to(dt).double()
                r["next_h"], r["next_rstd"] = kept / size(kept) * s["w_next"].double(), 1 / size(kept)[:, 0]
            return r
        dout, w = s["dout"].double(), s["w_post"].double()
        rs = s["rstd_post"].double()[:, None]
        u = b * dout * g * w
        r["dy"] = rs * u - y * rs ** 3 * torch.linalg.vecdot(u, y)[:, None] / H
        r["dw_post"] = (b * dout * g * y * rs).sum(0)
        r["dresidual"] = a * dout
        if s["gate"] is not None:
            dg = b * dout * y * rs * w * ((g - g * g) if c["sigmoid"] else 1.0)
            r["dgate"] = dg.sum(1) if c["gate"] == "token" else dg.sum(0) if c["gate"] == "channel" else dg
        rs, u = s["rstd_pre"].double()[:, None], s["dh"].double() * s["w_pre"].double()
        r["dx"] = rs * u - x * rs ** 3 * torch.linalg.vecdot(u, x)[:, None] / H + a * dout
        r["dw_pre"] = (s["dh"].double() * x * rs).sum(0)
        return r
    if c["op"] == "experts":
        K, N, E, P, ends = c["K"], c["N"], c["E"], c["T"] * c["k"], s["ends"]
        f = dict(device="cuda", dtype=torch.float64)
        if c["dir"] == "weights":
            dw = torch.zeros(E, N, K, **f)
            for e in range(E):
                dw[e] = torch.einsum("rn,rk->nk", s["dc"][ends[e]:ends[e + 1]].double(),
                                     s["a"][ends[e]:ends[e + 1]].double())
            return {"dw": dw}
        res = torch.zeros(P, K if c["dir"] == "rows" else N, **f)
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            if ends[e + 1] > ends[e]:
                res[at] = (torch.einsum("rn,nk->rk", s["dc"][at].double(), s["w"][e].double()) if c["dir"] == "rows"
                           else torch.einsum("rk,nk->rn", s["a"][at].double(), s["w"][e].double()))
        if c["dir"] == "rows":
            if not c["silu"]:
                return {"da": res}
            gate, up = s["gu"].double().chunk(2, dim=1)
            sg = torch.sigmoid(gate)
            return {"dgu": torch.cat([res * up * (sg + gate * sg * (1 - sg)), res * torch.nn.functional.silu(gate)], 1)}
        if not c["silu"]:
            return {"c": res}
        gate, up = res.chunk(2, dim=1)
        return {"gu": res, "h": gate * torch.sigmoid(gate) * up}
    grads = [x.double() for x in s["grads"]]
    if c["norm"] == "2":
        total = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(x) for x in grads]))
    else:
        total = max(x.abs().max() for x in grads)
    scale = min(1.0, s["max_norm"] / (float(total) + EPS))
    kinds = [t for _, t in _shapes(c)]
    return {"total": total, **{t: torch.cat([x.reshape(-1) * scale for x, u in zip(grads, kinds) if u == t])
                               for t in s["flat"]}}
