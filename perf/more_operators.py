"""The router of a mixture-of-experts layer and its experts in 4-bit floating point, case by case, in plain torch.

Three operators:

  router   routing in its training form: softmax or sigmoid scores, a bias for balance, groups of experts, the
           top-k with renormalised weights, a padding mask, the experts' loads with the balance and z losses, and
           the gradient of the logits;
  quant    microscaled 4-bit quantisation of rows (mxfp4: 32 values to a power-of-two scale; nvfp4: 16 values to
           an e4m3 scale, and a scale for each row), and the values that the codes stand for;
  experts  the experts' products on 4-bit rows and weights: one product, or the whole expert (SiLU(gate)*up of the first
           product, rounded to bf16 and quantised again, through the second), from 16-bit rows sorted by expert.

Where `own` is false, run() computes them in elementary torch operations, in 32 bits (what decides a rounding to 4 or 8 bits
or the choice of an expert: in 64); where it is true, through the package's entry points.  exact() is the same
in 64 bits from the definitions.

Shapes are those of the package's workloads (DeepSeek-V3-, Qwen3-30B-A3B- and Mixtral-shaped layers).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
GROUP = {"mxfp4": 32, "nvfp4": 16}


def _moe():
    import block_fp8_mixture_topk_gb300 as moe
    return moe


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of eight requests of a DeepSeek-V3-shaped layer: latency
        {"name": "router_decode", "op": "router", "dir": "forward", "T": 8, "E": 256, "k": 8, "dtype": "fp32",
         "scoring": "sigmoid", "bias": True, "groups": 8, "kept": 4, "group_score": "top2", "renorm": True, "scaling": 2.5,
         "padding": 0.0},
        # a training batch of the same layer: forward with the experts' loads, and the gradient
        {"name": "router_dsv3_train", "op": "router", "dir": "train", "T": 16384, "E": 256, "k": 8, "dtype": "fp32",
         "scoring": "sigmoid", "bias": True, "groups": 8, "kept": 4, "group_score": "top2", "renorm": True, "scaling": 2.5,
         "padding": 0.0},
        # a long padded batch of a Qwen3-30B-A3B-shaped layer, 16-bit logits
        {"name": "router_qwen3_train", "op": "router", "dir": "train", "T": 65536, "E": 128, "k": 8, "dtype": "bf16",
         "scoring": "softmax", "bias": False, "groups": 1, "kept": 1, "group_score": "top2", "renorm": True, "scaling": 1.0,
         "padding": 0.1},
        # the rows of eight decoding requests: latency
        {"name": "quant_decode", "op": "quant", "rows": 8, "K": 7168, "dtype": "bf16", "format": "nvfp4"},
        # the rows of a long Qwen3-30B-A3B-shaped batch, sorted by expert
        {"name": "quant_qwen3", "op": "quant", "rows": 131072, "K": 2048, "dtype": "bf16", "format": "mxfp4"},
        # a ragged batch held in 32 bits
        {"name": "quant_odd", "op": "quant", "rows": 5003, "K": 2880, "dtype": "fp32", "format": "nvfp4"},
        # one token through the eight experts of a Qwen3-30B-A3B-shaped layer: latency and the experts' weights
        {"name": "experts_one_token", "op": "experts", "dir": "mlp", "T": 1, "k": 8, "E": 128, "K": 2048, "I": 768,
         "dtype": "bf16", "format": "mxfp4", "skew": 0.0, "drop": 0.0},
        # 32 of a DeepSeek-V3-shaped layer's experts, the rows that a decoding batch sends them
        {"name": "experts_dsv3_decode", "op": "experts", "dir": "mlp", "T": 64, "k": 1, "E": 32, "K": 7168, "I": 2048,
         "dtype": "bf16", "format": "nvfp4", "skew": 0.0, "drop": 0.0},
        # a long Qwen3-30B-A3B-shaped prefill, skewed, some pairs dropped by a capacity limit
        {"name": "experts_qwen3", "op": "experts", "dir": "mlp", "T": 16384, "k": 8, "E": 128, "K": 2048, "I": 768,
         "dtype": "bf16", "format": "mxfp4", "skew": 1.2, "drop": 0.02},
        # a Mixtral-shaped prefill: few large experts
        {"name": "experts_mixtral", "op": "experts", "dir": "mlp", "T": 4096, "k": 2, "E": 8, "K": 4096, "I": 14336,
         "dtype": "bf16", "format": "nvfp4", "skew": 0.0, "drop": 0.0},
        # one product of a ragged batch for every token (a shared expert's second weight), 16-bit floats out
        {"name": "experts_shared", "op": "experts", "dir": "product", "T": 5003, "k": 1, "E": 1, "K": 2048, "I": 7168,
         "dtype": "fp16", "format": "mxfp4", "skew": 0.0, "drop": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "quant", "experts", "experts"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    form = rng.choice(["mxfp4", "nvfp4"])
    if op == "router":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = max(2, _log(rng, 8, 512) // groups) * groups
        kept = rng.randint(1, groups)
        return {"op": op, "dir": rng.choice(["forward", "train"]), "T": min(_log(rng, 1, 65536), (1 << 23) // E), "E": E,
                "k": rng.randint(1, min(8, E // groups * kept)), "dtype": dtype,
                "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6, "groups": groups, "kept": kept,
                "group_score": rng.choice(["top2", "max"]), "renorm": rng.random() < 0.7,
                "scaling": rng.choice([1.0, 2.5]), "padding": rng.choice([0.0, 0.1])}
    if op == "quant":
        rows = _log(rng, 1, 131072)
        return {"op": op, "rows": rows, "K": max(1, min(_log(rng, 32, 14336), (1 << 28) // rows) // 32) * 32,
                "dtype": dtype, "format": form}
    direction = rng.choice(["mlp", "product"])
    k = rng.choice([1, 2, 4, 8])
    E = _log(rng, k, 128)
    K = max(1, _log(rng, 64, 8192) // 32) * 32
    I = max(1, min(_log(rng, 64, 8192), (1 << 28) // (E * K)) // 32) * 32
    T = max(1, min(_log(rng, 1, 16384), int(4e11 / (k * K * I)), (1 << 28) // (k * max(K, I))))
    return {"op": op, "dir": direction, "T": T, "k": k, "E": E, "K": K, "I": I, "dtype": dtype if direction == "product" else
            rng.choice(["bf16", "fp16"]), "format": form, "skew": rng.choice([0.0, 1.2]), "drop": rng.choice([0.0, 0.05])}


def _touched(c):
    P, E = c["T"] * c["k"], c["E"]
    return int(round(E * (1 - (1 - 1 / E) ** P)))


def work(case):
    c, op = case, case["op"]
    if op == "router":
        T, E, k, b = c["T"], c["E"], c["k"], SIZES[c["dtype"]]
        forward = {"bytes": T * E * b + T * k * 8 + (4 * E if c["bias"] else 0) + (T if c["padding"] else 0),
                   "flops": T * E * 6}
        if c["dir"] == "forward":
            return forward
        # the loads out; the logits once more, the choice and its gradient in, the logits' gradient out
        return {"bytes": forward["bytes"] + 4 * E + 2 * T * E * b + T * k * 8, "flops": T * E * 18}
    bits = 4 + 8 / GROUP[c["format"]]
    if op == "quant":   # rows in, codes and scales out and in again, values out
        n = c["rows"] * c["K"]
        return {"bytes": int(n * (2 * SIZES[c["dtype"]] + 2 * bits / 8)), "flops": 4 * n}
    # rows in, touched weights in, results out
    P, K, I, b = c["T"] * c["k"], c["K"], c["I"], SIZES[c["dtype"]]
    if c["dir"] == "product":
        return {"bytes": int(b * (P * K + P * I) + _touched(c) * K * I * bits / 8), "flops": 2 * P * K * I}
    return {"bytes": int(b * 2 * P * K + _touched(c) * 3 * K * I * bits / 8), "flops": 6 * P * K * I}


# --------------------------------------------------------------------------------- 4-bit numbers
def _power(e):
    """2^e of whole numbers, in 64 bits, exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e2m1(a):
    """Nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code) to magnitudes."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return (torch.round(a / step) * step).clamp(max=6.0)


def _e4m3(a):
    """Nearest e4m3 number to magnitudes, as the values (saturating at 448)."""
    _, p = torch.frexp(a)
    step = _power(p.clamp(min=-5) - 4).to(a.dtype)   # 2^-9 below 2^-6
    return (torch.round(a / step) * step).clamp(max=448.0)


def _quantise(x, form):
    """(e2m1 values [R, K], scales [R, K/G], row scales [R] or None) of rows x."""
    R, K = x.shape
    g = x.double().reshape(R, -1, GROUP[form]) if form == "nvfp4" else x.float().reshape(R, -1, 32)
    a = g.abs()
    top = a.amax(2)
    if form == "mxfp4":
        m, p = torch.frexp(top)          # top = m 2^p, m in [1/2, 1): 2^(p-3) holds up to 6/8 2^p
        e = torch.where(top > 0, p - 3 + (m > 0.75), torch.full_like(p, -127)).clamp(-127, 127)
        scale, row = _power(e), None
        div = scale.to(g.dtype)
    else:
        row = (top.amax(1) / 2688).float()
        r = row.double()[:, None]
        scale = _e4m3(torch.where(r > 0, top / (6 * r), 0.0))
        div = scale * r
    q = torch.where(div[:, :, None] > 0, _e2m1(a / torch.where(div > 0, div, 1.0)[:, :, None]), 0.0)
    return (q * g.sign()).reshape(R, K), scale, row


def _values(q, scale, row):
    """The numbers that codes and scales stand for, in 32 bits."""
    v = (q.float().reshape(q.shape[0], scale.shape[1], -1) * scale.float()[:, :, None]).reshape(q.shape)
    return v if row is None else v * row[:, None]


_CODE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _codes(q):
    """e2m1 values [..., K] as codes, two to a byte, the first in the low half."""
    table = torch.tensor(_CODE, device=q.device, dtype=q.dtype)
    c = torch.searchsorted(table, q.abs().contiguous()).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _scale_bytes(scale, form):
    if form == "mxfp4":
        return (torch.frexp(scale)[1] + 126).to(torch.uint8)
    return scale.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _scale_tiles(s, form, gate_up):
    """Scale bytes [E, N, K/G] in the tiles that the products read: 128 rows by 256 columns, four scales to a word,
    rows 32 apart side by side; with gate_up, 16 gate rows and the 16 up rows of the same columns in turn."""
    E, N, C = s.shape
    if gate_up:
        s = s.reshape(E, 2, N // 32, 16, C).transpose(1, 2).reshape(E, N, C)
    words = 256 // GROUP[form] // 4
    nt, kb = -(-N // 128), -(-C // (4 * words))
    t = torch.zeros(E, nt * 128, kb * words * 4, dtype=torch.uint8, device=s.device)
    t[:, :N, :C] = s
    t = t.reshape(E, nt, 4, 32, kb, words, 4)               # row = 32 * (of 4) + (of 32)
    return t.permute(0, 1, 4, 5, 3, 2, 6).reshape(E, nt, kb, words * 512).contiguous()


def _weights(g, E, N, K, form, gate_up):
    """4-bit expert weights of normal values: what a program holds after loading them."""
    G = GROUP[form]
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // G, dtype=torch.uint8, device="cuda")
    total = torch.empty(E, device="cuda") if form == "nvfp4" else None
    for e in range(E):
        w = torch.randn(N, K, generator=g, device="cuda").mul_(K ** -0.5).reshape(N, K // G, G)
        top = w.abs().amax(2)
        if form == "nvfp4":
            total[e] = top.max() / 2688
            s = _e4m3(top / (6 * total[e])).clamp(min=2.0 ** -9)
            d = s * total[e]
        else:
            d = s = _power(torch.ceil(torch.log2(top / 6))).float()
        q = w.div_(d[:, :, None])
        codes[e] = _codes(_e2m1(q.abs()).copysign(q).reshape(N, K))
        scales[e] = _scale_bytes(s, form)
    return {"codes": codes, "scales": scales, "global": total, "tiles": _scale_tiles(scales, form, gate_up)}


def _scale_values(b, form, dtype):
    if form == "mxfp4":
        return _power(b.int() - 127).to(dtype)
    return b.view(torch.float8_e4m3fn).to(dtype)


def _weight_values(w, e, form, dtype):
    """Expert e's weights [N, K] from codes and scales."""
    table = torch.tensor(_CODE + [-v for v in _CODE], device="cuda", dtype=dtype)
    c = w["codes"][e]
    v = table[torch.stack([c & 15, c >> 4], 2).reshape(c.shape[0], -1).int()]
    s = _scale_values(w["scales"][e], form, dtype)
    v = (v.reshape(s.shape[0], s.shape[1], -1) * s[:, :, None]).reshape(v.shape)
    return v if w["global"] is None else v * w["global"][e].to(dtype)


# ----------------------------------------------------------------------------------------- inputs
def _offsets(g, c):
    """Rows of each expert [E+1] of a router with a popularity skew; the rows of dropped pairs are past the last."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits -= c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda"))
    ids = logits.topk(k, dim=1).indices
    if c["drop"]:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < c["drop"], E, ids)
    at = torch.sort(ids.reshape(-1)).values
    return torch.searchsorted(at, torch.arange(E + 1, device="cuda")).int()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "router":
        T, E = c["T"], c["E"]
        popular = torch.randn(E, generator=g, device="cuda").mul_(0.5)
        s["logits"] = (torch.randn(T, E, generator=g, device="cuda") + popular).to(dt)
        # a bias that many updates by 0.001 have brought towards balance
        s["bias"] = torch.round(popular * -40 + torch.randn(E, generator=g, device="cuda") * 4) * 0.001 if c["bias"] else None
        s["valid"] = torch.rand(T, generator=g, device="cuda") >= c["padding"] if c["padding"] else None
        s["dweights"] = torch.randn(T, c["k"], generator=g, device="cuda").mul_(0.1)
        s["balance"], s["z"] = 0.01, 0.001 if c["scoring"] == "softmax" else 0.0
    elif c["op"] == "quant":
        # activations: a few columns are larger than the others
        column = torch.exp(0.7 * torch.randn(c["K"], generator=g, device="cuda"))
        s["x"] = torch.randn(c["rows"], c["K"], generator=g, device="cuda").mul_(column).to(dt)
    else:
        K, I, E, P = c["K"], c["I"], c["E"], c["T"] * c["k"]
        s["offsets"] = _offsets(g, c)
        s["ends"] = s["offsets"].tolist()
        s["rows"] = torch.randn(P, K, generator=g, device="cuda", dtype=dt)
        if c["dir"] == "product":
            s["w"] = _weights(g, E, I, K, c["format"], False)
        else:
            s["w13"] = _weights(g, E, 2 * I, K, c["format"], True)
            s["w2"] = _weights(g, E, K, I, c["format"], False)
    return s


# -------------------------------------------------------------------------------------- plain form
def _choose(key, c):
    """Experts [T, k] of the largest keys, -1 where no expert with a finite key is left; ties: the lowest."""
    T, E = key.shape
    if c["groups"] > 1:
        by = key.reshape(T, c["groups"], -1)
        value = by.sort(dim=2, descending=True).values[:, :, :2].sum(2) if c["group_score"] == "top2" else by.amax(2)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(keep[:, :, None], by, -math.inf).reshape(T, E)
    top = key.sort(dim=1, descending=True, stable=True)
    return torch.where(top.values[:, :c["k"]] > -math.inf, top.indices[:, :c["k"]], -1)


def _router(s):
    c = s["case"]
    T, E, k, scaling = c["T"], c["E"], c["k"], c["scaling"]
    softmax = c["scoring"] == "softmax"
    wide = s["logits"].double()
    key = wide
    if c["bias"] or c["groups"] > 1:   # values next to a border: in 64 bits
        if softmax:
            u = torch.exp(wide - wide.amax(1, keepdim=True))
            key = u / u.sum(1, keepdim=True)
        else:
            key = 1 / (1 + torch.exp(-wide))
        if c["bias"]:
            key = key + s["bias"].double()
    ids = _choose(key, c)
    valid = s["valid"]
    if valid is not None:
        ids = torch.where(valid[:, None], ids, -1)
    l = s["logits"].float()
    m = l.amax(1, keepdim=True)
    if softmax:
        u = torch.exp(l - m)
        z = u.sum(1, keepdim=True)
        score, lse = u / z, (m + torch.log(z))[:, 0]
        share, phi = score, None
    else:
        score = 1 / (1 + torch.exp(-l))
        share, phi = score / score.sum(1, keepdim=True), 1 - score
    real, at = ids >= 0, ids.clamp(min=0)
    chosen = torch.where(real, score.gather(1, at), 0.0)
    q = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-37) if c["renorm"] else chosen
    r = {"ids": ids.int(), "weights": q * scaling}
    if c["dir"] == "forward":
        return r
    one = torch.zeros(T, E, device="cuda").scatter_add_(1, at, real.float())   # the choice
    r["counts"] = one.double().sum(0).int()
    live = torch.ones(T, device="cuda") if valid is None else valid.float()
    n = live.double().sum().float()
    f = r["counts"].float() * E / (k * n)
    r["balance"] = (f * (share * live[:, None]).sum(0)).sum() / n
    dshare = s["balance"] * f / n
    dl = share * (dshare - (share * dshare).sum(1, keepdim=True))
    if softmax:
        r["z"] = (lse.square() * live).sum() / n
        dl = dl + s["z"] * 2 * lse[:, None] / n * score
    else:
        dl = dl * phi
    dl = dl * live[:, None]
    dw = torch.where(real, s["dweights"], 0.0) * scaling
    if c["renorm"]:
        d = q * (dw - (q * dw).sum(1, keepdim=True))
        d = d if softmax else d * phi.gather(1, at)
        dl = dl.scatter_add(1, at, torch.where(real, d, 0.0))
    elif softmax:
        dense = torch.zeros(T, E, device="cuda").scatter_add_(1, at, dw)
        dl = dl + score * (dense - (q * dw).sum(1, keepdim=True))
    else:
        dl = dl.scatter_add(1, at, dw * q * phi.gather(1, at))
    r["dlogits"] = dl.to(s["logits"].dtype)
    return r


def _quant(s):
    q, scale, row = _quantise(s["x"], s["case"]["format"])
    return {"values": _values(q, scale, row).to(s["x"].dtype)}


def _product(rows, w, s):
    """4-bit rows (their values, in 32 bits) by every expert's weights; rows of no expert zero."""
    c = s["case"]
    ends = s["ends"]
    got = [rows[ends[e]:ends[e + 1]] @ _weight_values(w, e, c["format"], torch.float32).T
           for e in range(c["E"]) if ends[e + 1] > ends[e]]
    return torch.cat(got + [torch.zeros(rows.shape[0] - ends[-1], w["codes"].shape[1], device="cuda")])


def _experts(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    rows = _values(*_quantise(s["rows"], c["format"]))
    if c["dir"] == "product":
        return {"out": _product(rows, s["w"], s).to(dt)}
    gate, up = _product(rows, s["w13"], s).chunk(2, 1)
    h = (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    return {"out": _product(_values(*_quantise(h, c["format"])), s["w2"], s).to(dt)}


# ------------------------------------------------------------------------------------ entry points
def _own_router(s):
    moe, c = _moe(), s["case"]
    routing = moe.RoutingParams(scoring=c["scoring"], n_group=c["groups"], topk_group=c["kept"],
                                routed_scaling=c["scaling"], bias=s["bias"])
    train = c["dir"] == "train"
    r = moe.moe_router(s["logits"], c["k"], renormalize=c["renorm"], routing=routing, group_score=c["group_score"],
                       valid=s["valid"], losses=train)
    out = {"ids": r.ids, "weights": r.weights}
    if train:
        out["counts"], out["balance"] = r.counts, r.balance_loss
        if c["scoring"] == "softmax":
            out["z"] = r.z_loss
        out["dlogits"] = moe.moe_router_backward(s["logits"], r, s["dweights"], renormalize=c["renorm"], routing=routing,
                                                 balance_coef=s["balance"], z_coef=s["z"])
    return out


def _own_quant(s):
    moe = _moe()
    return {"values": moe.moe_fp4_dequant(moe.moe_fp4_quant(s["x"], s["case"]["format"]), s["x"].dtype)}


def _own_experts(s):
    moe, c = _moe(), s["case"]
    rows = moe.moe_fp4_quant(s["rows"], c["format"], s["offsets"])
    if c["dir"] == "product":
        w = s["w"]
        return {"out": moe.moe_fp4_expert_gemm(rows, w["codes"], w["tiles"], w["global"], dtype=DTYPES[c["dtype"]])}
    w, w2 = s["w13"], s["w2"]
    h = moe.moe_fp4_expert_gemm_silu_mul_quant(rows, w["codes"], w["tiles"], w["global"])
    return {"out": moe.moe_fp4_expert_gemm(h, w2["codes"], w2["tiles"], w2["global"], dtype=DTYPES[c["dtype"]])}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"router": _own_router, "quant": _own_quant, "experts": _own_experts}[op](state)
    return {"router": _router, "quant": _quant, "experts": _experts}[op](state)


# ------------------------------------------------------------------------------------- in 64 bits
def _exact_router(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].double()
    score = torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l)
    key = l if not c["bias"] and c["groups"] == 1 else score + (0 if s["bias"] is None else s["bias"].double())
    G = c["groups"]
    if G > 1:   # a group's place: the groups before it, or equal and of a lower number
        by = key.reshape(T, G, E // G)
        v = by.amax(2) if c["group_score"] == "max" else by.topk(min(2, E // G), dim=2).values.sum(2)
        lower = torch.arange(G, device="cuda")
        ahead = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (lower[None, :] < lower[:, None]))
        key = key.masked_fill((ahead.sum(2) >= c["kept"]).repeat_interleave(E // G, 1), -math.inf)
    picked, left = [], key.clone()
    for _ in range(k):
        best = (left == left.amax(1, keepdim=True)).int().argmax(1)     # the first of the largest
        picked.append(best)
        left.scatter_(1, best[:, None], -math.inf)
    ids = torch.stack(picked, 1)
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]
    lw = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, ids, s["dweights"].double()) * c["scaling"]
    S = torch.zeros(T, E, dtype=torch.bool, device="cuda").scatter_(1, ids, True)
    w = torch.where(S, score, 0.0)
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    r = {"ids": torch.where(live[:, None], ids, -1).int(),
         "weights": torch.where(live[:, None], w.gather(1, ids), 0.0) * c["scaling"]}
    if c["dir"] == "forward":
        return r
    n = live.sum()
    counts = (S & live[:, None]).sum(0)
    r["counts"] = counts.int()
    share = score / score.sum(1, keepdim=True)
    f = counts.double() * E / (k * n)
    r["balance"] = (share[live].mean(0) * f).sum()
    # gradients by the scores, then through them
    dscore = torch.zeros_like(score)
    total = score.sum(1, keepdim=True)
    df = s["balance"] * f / n
    dscore += df / total - (score * df).sum(1, keepdim=True) / total.square()
    if c["renorm"]:
        z = torch.where(S, score, 0.0).sum(1, keepdim=True)
        dscore += torch.where(S, lw / z - (lw * w).sum(1, keepdim=True) / z, 0.0)
    else:
        dscore += lw
    if c["scoring"] == "softmax":
        lse = torch.logsumexp(l, 1)
        r["z"] = lse[live].square().mean()
        dl = score * (dscore - (score * dscore).sum(1, keepdim=True)) + s["z"] * 2 * lse[:, None] * score / n
    else:
        dl = dscore * score * (1 - score)
    r["dlogits"] = dl * live[:, None]
    return r


def _exact_quant(x, form):
    """The values of x in 4 bits: each number's nearest by the borders between them."""
    R, K = x.shape
    G = GROUP[form]
    v = x.double().reshape(R, K // G, G)
    top = v.abs().amax(2, keepdim=True)
    if form == "mxfp4":
        d = _power(torch.arange(-127, 128, device="cuda"))      # the first scale that holds the largest
        d = d[torch.searchsorted(d, (top / 6).contiguous()).clamp(max=254)]
    else:
        row = (top.amax(1, keepdim=True) / 2688).float().double()
        table = torch.arange(0, 127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        b = _nearest((top / (6 * row)).nan_to_num(0.0), table)
        d = b * row
    table = torch.tensor(_CODE, dtype=torch.float64, device="cuda")
    q = _nearest((v.abs() / d).nan_to_num(0.0, 0.0, 0.0), table)
    return (q * d * v.sign()).reshape(R, K)


def _nearest(a, table):
    """Nearest entry of an ascending table, ties to the even index."""
    hi = torch.searchsorted(table, a.contiguous()).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    return table[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "router":
        return _exact_router(s)
    if c["op"] == "quant":
        return {"values": _exact_quant(s["x"], c["format"])}
    form, P = c["format"], c["T"] * c["k"]

    def product(rows, w):
        out = torch.zeros(P, w["codes"].shape[1], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            lo, hi = s["ends"][e], s["ends"][e + 1]
            if hi > lo:
                out[lo:hi] = rows[lo:hi] @ _weight_values(w, e, form, torch.float64).T
        return out

    rows = _exact_quant(s["rows"], form)
    if c["dir"] == "product":
        return {"out": product(rows, s["w"])}
    gate, up = product(rows, s["w13"]).chunk(2, 1)
    h = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)
    return {"out": product(_exact_quant(h, form), s["w2"])}
