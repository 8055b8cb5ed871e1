"""The training router against 64-bit values: choice, weights, loads and losses, and the gradient of the logits."""
import dataclasses
import math

import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from train_testutil import DTYPES, check, gen, ids_of, offset_copy, status, status_clear, strided_copy

pytestmark = pytest.mark.gpu


@dataclasses.dataclass
class Case:
    T: int
    E: int
    k: int
    scoring: str = "softmax"
    bias: str = ""          # "", "zero", "steps" (multiples of 0.001), "large"
    groups: int = 1
    kept: int = 1
    score: str = "top2"
    renorm: bool = True
    scaling: float = 1.0
    dtype: torch.dtype = torch.float32
    padding: float = 0.0
    spread: float = 1.0

    def __str__(self):
        return "-".join(str(v).replace("torch.", "") for v in dataclasses.astuple(self))


CASES = [
    Case(1, 1, 1), Case(3, 8, 2), Case(5, 8, 8, "sigmoid"), Case(33, 33, 4, dtype=torch.bfloat16),
    Case(100, 256, 8, "sigmoid", "steps", 8, 4, scaling=2.5), Case(257, 256, 8, "sigmoid", "steps", 8, 4, dtype=torch.bfloat16),
    Case(64, 128, 8, dtype=torch.bfloat16, padding=0.2), Case(64, 128, 8, dtype=torch.float16, renorm=False, scaling=1.7),
    Case(70, 160, 6, "softmax", "", 8, 3, "max", renorm=False, scaling=16.0), Case(70, 160, 6, "softmax", "steps", 8, 3, "top2"),
    Case(40, 60, 5, "sigmoid", "large", 6, 2, "max", renorm=False), Case(40, 60, 5, "sigmoid", "", 12, 7, "top2", False),
    Case(90, 512, 32, "softmax", "zero"), Case(90, 1024, 32, "sigmoid", "steps", 32, 5, dtype=torch.bfloat16),
    Case(2000, 64, 2, "softmax", "steps", padding=0.5, renorm=False), Case(5000, 16, 4, "sigmoid", "steps", dtype=torch.float16),
    Case(20, 300, 7, "sigmoid", "steps", 3, 2), Case(77, 1000, 10, "softmax", "steps", 10, 3, renorm=False),
    Case(50, 32, 4, "softmax", spread=30.0), Case(50, 32, 4, "sigmoid", spread=60.0), Case(50, 32, 4, "sigmoid", "large", spread=60.0),
    Case(60, 96, 3, "softmax", "steps", 3, 1, "max", dtype=torch.bfloat16, padding=0.3),
]


def inputs(c, seed, device="cuda"):
    g = gen(seed)
    logits = (torch.randn(c.T, c.E, generator=g) * c.spread).to(c.dtype)
    bias = {"": None, "zero": torch.zeros(c.E), "steps": torch.randint(-40, 41, (c.E,), generator=g) * 0.001,
            "large": torch.randn(c.E, generator=g)}[c.bias]
    valid = torch.rand(c.T, generator=g) >= c.padding if c.padding else None
    to = lambda t: None if t is None else t.to(device)  # noqa: E731
    return to(logits), to(bias), to(valid), torch.randn(c.T, c.k, generator=g).to(device)


def routing(c, bias):
    return moe.RoutingParams(scoring=c.scoring, n_group=c.groups, topk_group=c.kept, routed_scaling=c.scaling, bias=bias)


def reference(c, logits, bias, valid, dweights=None, balance=0.0, z=0.0):
    """Everything in 64 bits, on the CPU; the gradient by differentiating the formulas."""
    l = logits.double().cpu().requires_grad_()
    T, E, k = c.T, c.E, c.k
    masked = ~torch.isfinite(l.detach())
    lm = torch.where(masked, -math.inf, l)
    softmax = c.scoring == "softmax"
    alive = ~masked.all(1)
    if valid is not None:
        alive &= valid.cpu().bool()
    safe = torch.where(alive[:, None], lm, 0.0)
    # (through its logarithm, whose derivative sigmoid(-l) keeps its digits where 1 - sigmoid(l) has none left)
    score = torch.softmax(safe, 1) if softmax else torch.exp(torch.nn.functional.logsigmoid(safe))
    key = (score if bias is not None or c.groups > 1 else safe).detach()
    if bias is not None:
        key = key + bias.double().cpu()
    elif c.groups > 1 and c.score == "max":
        key = safe.detach()
    key = torch.where(masked, -math.inf, key)
    if c.groups > 1:
        by = key.reshape(T, c.groups, -1)
        top = by.sort(dim=2, descending=True).values[:, :, :1 if c.score == "max" else 2]
        value = torch.where(top == -math.inf, 0.0, top).sum(2).masked_fill((by == -math.inf).all(2), -math.inf)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, :c.kept]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        key = by.masked_fill(~keep[:, :, None], -math.inf).reshape(T, E)
    top = key.sort(dim=1, descending=True, stable=True)
    ids = torch.where((top.values > -math.inf) & alive[:, None], top.indices, -1)[:, :k]
    real = ids >= 0
    s = torch.where(real, score.gather(1, ids.clamp(min=0)), 0.0)
    if c.renorm:   # in the logarithm, so that scores that vanish keep their ratios
        at = safe.gather(1, ids.clamp(min=0))
        log = torch.where(real, at if softmax else torch.nn.functional.logsigmoid(at), -math.inf)
        q = torch.softmax(torch.where(real.any(1, keepdim=True), log, 0.0), 1) * real
    else:
        q = s
    w = q * c.scaling
    n = int(alive.sum())
    counts = torch.bincount(ids[real], minlength=E)
    total = score.sum(1, keepdim=True)
    share = torch.where(alive[:, None], score / torch.where(alive[:, None], total, 1.0), 0.0)
    f = counts.double() * E / (k * max(n, 1))
    bal = (f * share.sum(0)).sum() / max(n, 1)
    lse = torch.where(alive, torch.logsumexp(safe, 1), 0.0)
    zl = lse.square().sum() / max(n, 1)
    out = dict(ids=ids, w=w.detach(), counts=counts, n=n, balance=bal.detach(), z=zl.detach(), lse=lse.detach(),
               span=max(1.0, float(torch.where(torch.isfinite(lm) & alive[:, None], safe.max(1, keepdim=True).values - safe, 0.0).detach().max())))
    if dweights is not None:
        dw = torch.where(real, dweights.double().cpu(), 0.0)
        loss = (dw * w).sum() + balance * bal + (z * zl if softmax else 0.0)
        out["dlogits"] = torch.autograd.grad(loss, l)[0].nan_to_num(0.0)
        # magnitudes that meet in each value
        phi = torch.ones_like(score) if softmax else torch.sigmoid(-safe)
        g = dw.abs() * c.scaling
        h = balance * f / max(n, 1)
        size = share * (h.abs() + (share * h).sum(1, keepdim=True)) * phi
        if softmax:
            size = size + score * z * 2 * lse.abs()[:, None] / max(n, 1)
        inner = (q * g).sum(1, keepdim=True)
        if softmax and not c.renorm:
            size = size + score * inner
        own = q * (g + inner) * phi.gather(1, ids.clamp(min=0))
        out["size"] = (size * alive[:, None]).scatter_add(1, ids.clamp(min=0), torch.where(real, own, 0.0)).detach()
        # what scores, shares, phi and weights are multiplied by
        out["factor"] = (h.abs().max() + z * 2 * lse.abs()[:, None] / max(n, 1) + g.amax(1, keepdim=True)).detach()
    return out


def roundings(c, span):
    """fp32 half-steps of a score or weight: expf and a quotient 2 ulp (4 half-steps) each, twice (the score, its sum), the
    distance to the largest logit rounded once, a sum over a lane's and a warp's experts, a few products."""
    return 30 + 2 * span + max(1, c.E // 32) + 5


@pytest.mark.parametrize("c", CASES, ids=str)
def test_choice_weights_and_loads(c):
    logits, bias, valid, _ = inputs(c, 1)
    ref = reference(c, logits, bias, valid)
    status_clear()
    plain = moe.moe_router(logits, c.k, c.renorm, routing(c, bias), c.score, valid)
    r = moe.moe_router(logits, c.k, c.renorm, routing(c, bias), c.score, valid, losses=True)
    assert plain.counts is None and torch.equal(plain.ids, r.ids) and torch.equal(plain.weights, r.weights)
    assert torch.equal(r.ids.cpu().long(), ref["ids"])
    n = roundings(c, ref["span"])
    check(r.weights, ref["w"], ref["w"], n, "weights")
    assert torch.equal(r.counts.cpu().long(), ref["counts"]) and int(r.tokens) == ref["n"]
    # a sum over tokens: a warp's (T / 2432 and one), a block's 8, the blocks' 38 at most and their 16
    check(r.balance_loss, ref["balance"], ref["balance"], 2 * n + c.T / 2432 + 80, "balance")
    if c.scoring == "softmax":
        m = logits.double().cpu().abs().max()
        lse = ref["lse"].abs()
        size = (2 * lse * (m + math.log(c.E) + 1) + lse.square()).sum() / max(ref["n"], 1)
        check(r.z_loss, ref["z"], size, n + c.T / 2432 + 80, "z")
    else:
        assert r.z_loss is None
    assert status() == 0


@pytest.mark.parametrize("losses", [False, True])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_gradient(c, losses):
    logits, bias, valid, dw = inputs(c, 2)
    balance, z = (0.7 * c.T, 0.3 * c.T if c.scoring == "softmax" else 0.0) if losses else (0.0, 0.0)
    ref = reference(c, logits, bias, valid, dw, balance, z)
    r = moe.moe_router(logits, c.k, c.renorm, routing(c, bias), c.score, valid, losses=losses)
    got = moe.moe_router_backward(logits, r, dw, c.renorm, routing(c, bias), balance, z)
    assert got.dtype == c.dtype
    # four factors with the error of a score or weight in a term (q, the inner sum, phi, the loads' factor); a factor that
    # underflows is off by up to 2^-149 whatever its size, which is multiplied by the others (h and the mean of h, ...)
    n = 4 * roundings(c, ref["span"])
    check(got, ref["dlogits"], ref["size"] + 4 * 2.0 ** -149 * 2 * ref["factor"] / (n * 2.0 ** -24), n, "dlogits")


@pytest.mark.parametrize("c", [CASES[4], CASES[7], CASES[8], CASES[15]], ids=str)
def test_gradient_against_differences(c):
    """Differences of the fp64 formulas at the kernel's choice."""
    c = dataclasses.replace(c, T=6, dtype=torch.float32)
    logits, bias, valid, dw = inputs(c, 3)
    r = moe.moe_router(logits, c.k, c.renorm, routing(c, bias), c.score, valid)
    got = moe.moe_router_backward(logits, r, dw, c.renorm, routing(c, bias)).double().cpu()
    ids = r.ids.long().cpu()

    def loss(l):
        s = torch.softmax(l, 1) if c.scoring == "softmax" else torch.sigmoid(l)
        w = s.gather(1, ids)
        w = w / w.sum(1, keepdim=True) if c.renorm else w
        return (w * c.scaling * dw.double().cpu()).sum(1)

    l = logits.double().cpu()
    eps = 1e-5
    for e in torch.cat([ids[0], torch.arange(0, c.E, 17)]).unique().tolist():
        d = torch.zeros_like(l)
        d[:, e] = eps
        diff = (loss(l + d) - loss(l - d)) / (2 * eps)
        # the third derivative is below 2 scaling |dw|, the fp32 gradient's error below 1e-5 of that
        assert ((diff - got[:, e]).abs() <= 3e-5 * c.scaling * dw.double().cpu().abs().sum(1)).all()


def test_equal_keys_take_the_lower_expert():
    for dtype in DTYPES:
        for scoring in ("softmax", "sigmoid"):
            for bias in (None, torch.zeros(64, device="cuda"), torch.full((64,), 0.25, device="cuda")):
                rp = moe.RoutingParams(scoring=scoring, bias=bias)
                r = moe.moe_router(torch.zeros(5, 64, dtype=dtype, device="cuda"), 6, routing=rp)
                assert r.ids.tolist() == [[0, 1, 2, 3, 4, 5]] * 5
                assert torch.allclose(r.weights, torch.full_like(r.weights, 1 / 6), rtol=1e-6)
                rp.n_group, rp.topk_group = 8, 2
                r = moe.moe_router(torch.zeros(5, 64, dtype=dtype, device="cuda"), 10, routing=rp)
                assert r.ids.tolist() == [list(range(10))] * 5


def test_keys_closer_than_their_fp32_error():
    """Sums of score and bias that differ in the 9th digit: the order is that of the real numbers."""
    g = gen(5)
    for scoring in ("softmax", "sigmoid"):
        T, E, k = 200, 64, 8
        l = torch.randn(T, E, generator=g)
        # a bias that makes the keys of token t's experts nearly equal: the same logits for all tokens
        l[:] = l[0]
        l += torch.randn(T, E, generator=g) * 1e-7
        s = torch.softmax(l[0].double(), 0) if scoring == "softmax" else torch.sigmoid(l[0].double())
        bias = (1.0 - s).float()
        for groups, kept in ((1, 1), (8, 3)):
            c = Case(T, E, k, scoring, "given", groups, kept)
            ref = reference(c, l, bias, None)
            r = moe.moe_router(l.cuda(), k, routing=routing(c, bias.cuda()))
            assert torch.equal(r.ids.cpu().long(), ref["ids"]), (scoring, groups)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_logits(scoring, dtype):
    """Experts at -inf, a token with fewer than k left, with none, with NaN and +inf; the type's lowest value is a logit."""
    g = gen(6)
    for c in (Case(12, 64, 4, scoring, dtype=dtype), Case(12, 64, 4, scoring, "steps", 8, 2, dtype=dtype),
              Case(12, 60, 4, scoring, "", 6, 2, renorm=False, dtype=dtype)):
        l = torch.randn(c.T, c.E, generator=g).to(dtype)
        l[0, 1:] = -math.inf
        l[1] = -math.inf
        l[2, 2:] = -math.inf
        l[3, ::2] = -math.inf
        l[4, 5:] = torch.finfo(dtype).min
        l[5] = torch.finfo(dtype).min
        bias = torch.randint(-40, 41, (c.E,), generator=g) * 0.001 if c.bias else None
        dw = torch.randn(c.T, c.k, generator=g)
        z = 0.5 if scoring == "softmax" else 0.0
        # a logit of finfo.min makes lse^2 overflow fp32: those two tokens without losses
        for rows, coefs in ((slice(0, 12), (0.0, 0.0)), (slice(6, 12), (0.9, z))):
            cc = dataclasses.replace(c, T=len(range(12)[rows]))
            part = l[rows].clone()
            if coefs[0]:
                part[0, 1:], part[1], part[2, 2:] = -math.inf, -math.inf, -math.inf
            ref = reference(cc, part, bias, None, dw[rows], *coefs)
            x = part.cuda()
            rp = routing(cc, None if bias is None else bias.cuda())
            status_clear()
            r = moe.moe_router(x, c.k, c.renorm, rp, c.score, losses=bool(coefs[0]))
            assert torch.equal(r.ids.cpu().long(), ref["ids"])
            span = min(ref["span"], 100.0)   # scores e^-100 of the largest are below any half-step
            n = roundings(cc, span)
            check(r.weights, ref["w"], ref["w"], n, "weights")
            got = moe.moe_router_backward(x, r, dw[rows].cuda().contiguous(), c.renorm, rp, *coefs)
            check(got, ref["dlogits"], ref["size"], 4 * n, "dlogits")
            assert status() == 0
            # what is not a number is reported and counts as -inf
            y = x.clone()
            y[2, 7] = float("nan")
            y[2, 9] = float("inf")
            r2 = moe.moe_router(y, c.k, c.renorm, rp, c.score, losses=bool(coefs[0]))
            assert status() == 0x10
            y[2, 7] = y[2, 9] = -math.inf
            r3 = moe.moe_router(y, c.k, c.renorm, rp, c.score, losses=bool(coefs[0]))
            assert torch.equal(r2.ids, r3.ids) and torch.equal(r2.weights, r3.weights) and status() == 0


def test_strides_and_addresses():
    c = Case(50, 128, 8, "softmax", "", renorm=False)
    for dtype in DTYPES:
        logits, _, _, dw = inputs(dataclasses.replace(c, dtype=dtype), 7)
        r = moe.moe_router(logits, 8, False, losses=True)
        d = moe.moe_router_backward(logits, r, dw, False, balance_coef=1.0, z_coef=1.0)
        for y in (offset_copy(logits), strided_copy(logits, 1), strided_copy(logits, 8, 8), strided_copy(logits, 3, 2)):
            r2 = moe.moe_router(y, 8, False, losses=True)
            assert torch.equal(r.ids, r2.ids) and torch.equal(r.weights, r2.weights)
            assert torch.equal(r.balance_loss, r2.balance_loss) and torch.equal(r.z_loss, r2.z_loss)
            assert torch.equal(moe.moe_router_backward(y, r2, dw, False, balance_coef=1.0, z_coef=1.0), d)


def test_no_tokens_and_all_padded():
    r = moe.moe_router(torch.empty(0, 16, device="cuda"), 2, losses=True)
    assert r.ids.shape == (0, 2) and int(r.tokens) == 0 and float(r.balance_loss) == 0 and float(r.z_loss) == 0
    assert r.counts.tolist() == [0] * 16
    x = torch.randn(9, 16, device="cuda")
    r = moe.moe_router(x, 2, valid=torch.zeros(9, dtype=torch.bool, device="cuda"), losses=True)
    assert (r.ids == -1).all() and (r.weights == 0).all() and int(r.tokens) == 0 and float(r.balance_loss) == 0
    d = moe.moe_router_backward(x, r, torch.ones(9, 2, device="cuda"), balance_coef=1.0, z_coef=1.0)
    assert (d == 0).all()


def test_results_repeat_and_replay():
    c = Case(3000, 256, 8, "sigmoid", "steps", 8, 4, dtype=torch.bfloat16, padding=0.1)
    logits, bias, valid, dw = inputs(c, 8)

    def step():
        r = moe.moe_router(logits, c.k, True, routing(c, bias), "top2", valid, losses=True)
        return [r.ids, r.weights, r.counts, r.balance_loss, moe.moe_router_backward(logits, r, dw, True, routing(c, bias), 0.1)]

    want = step()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.current_stream().wait_stream(side)
    logits.copy_(inputs(c, 9)[0])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_bias_update():
    counts = torch.tensor([10, 0, 5, 5, 5, 5, 4, 6], dtype=torch.int32, device="cuda")
    bias = torch.zeros(8, device="cuda")
    moe.moe_router_update_bias(bias, counts, 0.001)
    assert torch.equal(bias, torch.tensor([-1, 1, 0, 0, 0, 0, 1, -1], device="cuda") * 0.001)
    counts = torch.randint(0, 2 ** 30, (1000,), generator=gen(10), dtype=torch.int32).cuda()
    bias = torch.zeros(1000, device="cuda")
    moe.moe_router_update_bias(bias, counts, 1.0)
    wide = counts.long().cpu()
    assert torch.equal(bias.cpu(), torch.sign(wide.sum() - wide * 1000).float())


def test_agrees_with_the_layers_router():
    """Where moe_route_topk takes the call, both choose the same experts with the same weights."""
    g = gen(11)
    for rp, E, k in ((None, 128, 8), (moe.RoutingParams(scoring="sigmoid", n_group=8, topk_group=4, routed_scaling=2.5,
                                                         bias=(torch.randn(256, generator=g) * 0.1).cuda()), 256, 8)):
        x = torch.randn(500, E, generator=g).cuda()
        ids, w = moe.moe_route_topk(x, k, True, rp)
        r = moe.moe_router(x, k, True, rp)
        assert torch.equal(ids, r.ids)
        assert ((w - r.weights).abs() <= w * 60 * 2.0 ** -24).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [40, 6000])
def test_bias_masks_experts(T, scoring):
    """A bias of -inf takes its expert out of the choice and of its group's value, not out of the shares."""
    g = gen(12)
    for E, groups, kept in ((64, 1, 1), (64, 8, 3), (60, 6, 2)):
        l = torch.randn(T, E, generator=g)
        bias = torch.randint(-40, 41, (E,), generator=g) * 0.001
        gone = torch.zeros(E, dtype=torch.bool)
        gone[::3] = True
        c = Case(T, E, 4, scoring, "given", groups, kept)
        ref = reference(c, torch.where(gone, -math.inf, l), bias, None)
        r = moe.moe_router(l.cuda(), 4, routing=routing(c, torch.where(gone, -math.inf, bias).cuda()), losses=True)
        # (softmax keys shift with the masked experts' share of the sum: compare where the reference has it too)
        if scoring == "sigmoid":
            assert torch.equal(r.ids.cpu().long(), ref["ids"])
        assert not gone[r.ids.cpu().long()].any()
        ref = reference(dataclasses.replace(c, groups=1), l, torch.where(gone, -1e30, bias), None)
        if groups == 1:
            assert torch.equal(r.ids.cpu().long(), ref["ids"])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(300, 64), (6000, 64), (6000, 200)])
def test_tokens_of_masked_experts_only(T, E, scoring):
    """A token whose logits above -inf are all of masked experts chooses none: it is not counted, has no share in the losses and
    no gradient."""
    g = gen(14)
    l = torch.randn(T, E, generator=g)
    bias = torch.zeros(E)
    bias[E // 2:] = -math.inf
    none = torch.rand(T, generator=g) < 0.2
    l[none, :E // 2] = -math.inf
    rp = moe.RoutingParams(scoring, bias=bias.cuda())
    r = moe.moe_router(l.cuda(), 4, routing=rp, losses=True)
    rest = moe.moe_router(l[~none].cuda(), 4, routing=rp, losses=True)
    assert (r.ids.cpu()[none] == -1).all() and (r.weights.cpu()[none] == 0).all()
    assert torch.equal(r.ids.cpu()[~none], rest.ids.cpu()) and torch.equal(r.counts, rest.counts)
    assert int(r.tokens) == int(rest.tokens) == int((~none).sum())
    # sums of at most T positive terms in another order
    tol = 2 * T * 2.0 ** -24
    assert abs(float(r.balance_loss) - float(rest.balance_loss)) <= tol * float(rest.balance_loss)
    if scoring == "softmax":
        assert abs(float(r.z_loss) - float(rest.z_loss)) <= tol * float(rest.z_loss)
    dl = moe.moe_router_backward(l.cuda(), r, torch.ones_like(r.weights), routing=rp, balance_coef=0.1,
                                 z_coef=0.1 if scoring == "softmax" else 0.0)
    assert (dl.cpu()[none] == 0).all() and torch.isfinite(dl).all()


def test_many_tokens():
    """Logits past 2^31 elements: the last tokens come out as they do alone."""
    T, E = 8_500_000, 256
    x = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    tail = x[-500:].clone()
    rp = moe.RoutingParams("sigmoid", n_group=8, topk_group=4)
    r = moe.moe_router(x, 8, routing=rp, losses=True)
    one = moe.moe_router(tail, 8, routing=rp)
    assert torch.equal(r.ids[-500:], one.ids) and torch.equal(r.weights[-500:], one.weights)
    assert int(r.tokens) == T and int(r.counts.long().sum()) == 8 * T
    dw = torch.ones(T, 8, device="cuda")
    dw[:, ::2] = 0.5
    d = moe.moe_router_backward(x, r, dw, routing=rp)
    assert torch.equal(d[-500:], moe.moe_router_backward(tail, one, dw[-500:].contiguous(), routing=rp))


@pytest.mark.parametrize("E", [24, 56, 100, 128])
def test_many_and_few_tokens_agree(E):
    """Four tokens to a warp and one choose and weigh alike, and gather the same loads."""
    for scoring, bias in (("softmax", False), ("sigmoid", True)):
        g = gen(13)
        x = torch.randn(9000, E, generator=g).bfloat16().cuda()
        rp = moe.RoutingParams(scoring, bias=(torch.randint(-40, 41, (E,), generator=g) * 0.001).cuda() if bias else None)
        valid = (torch.rand(9000, generator=g) > 0.1).cuda()
        r = moe.moe_router(x, 6, routing=rp, valid=valid, losses=True)
        parts = [moe.moe_router(x[i:i + 3000], 6, routing=rp, valid=valid[i:i + 3000], losses=True) for i in range(0, 9000, 3000)]
        assert torch.equal(r.ids, torch.cat([p.ids for p in parts]))
        assert torch.equal(r.counts, sum(p.counts for p in parts)) and int(r.tokens) == sum(int(p.tokens) for p in parts)
        w = torch.cat([p.weights for p in parts])
        assert ((r.weights - w).abs() <= 30 * 2.0 ** -24 * w).all()   # sums of the same terms in another order
