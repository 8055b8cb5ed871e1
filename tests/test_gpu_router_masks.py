"""The training router's masks and borders: experts masked by their bias, keys that meet in 64 bits, scores that vanish, and the same
decisions where four tokens share a warp."""
import math

import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
import test_gpu_router as base
from train_testutil import gen

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------- the balancing bias
@pytest.mark.parametrize("E", [1, 2, 7, 32, 33, 256, 1000, 1024])
def test_bias_update_leaves_masked_experts_out(E):
    """The mean is that of the experts that can be chosen; masked ones stay masked, whatever their counts."""
    g = gen(E)
    for share in (0.0, 0.3, 0.9, 1.0):
        masked = torch.rand(E, generator=g) < share
        counts = torch.randint(0, 2 ** 20, (E,), generator=g, dtype=torch.int32)
        bias = torch.where(masked, -math.inf, torch.randint(-40, 41, (E,), generator=g) * 0.25)
        got = bias.cuda()
        moe.moe_router_update_bias(got, counts.cuda(), 0.5)
        able = counts.long()[~masked]
        want = bias.clone()
        want[~masked] += 0.5 * torch.sign(able.sum() - able * len(able)).float()
        assert torch.equal(got.cpu(), want)


def test_bias_update_keeps_an_even_load_of_the_unmasked():
    """Half of the experts masked and the rest loaded evenly: nothing moves, step after step."""
    E, g = 64, gen(1)
    bias = torch.zeros(E)
    bias[::2] = -math.inf
    bias = bias.cuda()
    want = bias.clone()
    counts = torch.zeros(E, dtype=torch.int32)
    counts[1::2] = 17
    for _ in range(5):
        moe.moe_router_update_bias(bias, counts.cuda(), 0.001)
    assert torch.equal(bias, want)
    # and an expert between the two means is pushed up
    counts[1] = 12
    counts[3] = 22
    moe.moe_router_update_bias(bias, counts.cuda(), 0.001)
    assert bias[1] > 0 and bias[3] < 0 and (bias[5::2] == 0).all()
    r = moe.moe_router(torch.randn(300, E, generator=g).cuda(), 4, routing=moe.RoutingParams("sigmoid", bias=bias), losses=True)
    assert (r.counts[::2] == 0).all()


# ---------------------------------------------------------------------------- keys nearer than fp32 tells
def score64(l, scoring):
    l = l.double()
    return torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)


def choice64(l, bias, scoring, k):
    """The k largest fp64 keys, ties to the lower expert."""
    return (score64(l, scoring) + bias.double()).sort(dim=1, descending=True, stable=True).indices[:, :k]


@pytest.mark.parametrize("T", [300, 6000])
@pytest.mark.parametrize("copies", [2, 3, 20, 40])
@pytest.mark.parametrize("above", [0, 3, 7])
def test_a_near_key_behind_equal_ones(above, copies, T):
    """At the border of the choice lie experts of one logit and one bias, and behind them one whose key is as near as fp32 tells, of
    another logit and bias: it is chosen where its real key is larger."""
    g, E = gen(2), 64
    for last in (True, False):
        bias = torch.full((E,), -3.0)
        order = torch.randperm(E, generator=g)
        alike = order[:copies].sort().values
        other = E - 1 if last else 0
        alike = alike[alike != other]
        bias[alike], bias[other] = 0.125, 0.375
        top = torch.tensor([e for e in order.tolist() if e != other and e not in alike.tolist()][:above], dtype=torch.long)
        bias[top] = 4.0
        l = torch.randn(T, E, generator=g)
        x = 0.5 + torch.rand(T, generator=g)
        s = torch.sigmoid(x.double())
        l[:, alike] = x[:, None]
        want = s + 0.125 - 0.375
        l[:, other] = torch.log(want / (1 - want)).float()   # the same key but for the rounding of its logit: 2^-26 or so
        for k in (above + 1, above + 2):
            ref = choice64(l, bias, "sigmoid", k)
            r = moe.moe_router(l.cuda(), k, routing=moe.RoutingParams("sigmoid", bias=bias.cuda()))
            assert torch.equal(r.ids.cpu().long(), ref), (last, k)


# ------------------------------------------------------------------------- keys that are equal in fp64
def routes(T):
    """Sizes that reach the warp-a-token and the four-tokens-a-warp kernel."""
    return ((300, 64), (T, 64), (T, 128), (T, 256))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [0.0, 0.375, -2.0])
def test_one_bias_for_all_orders_as_the_logits(scoring, value):
    """Scores that are 1 to fp64's last bit, that vanish in it or in the bias: with one bias for all the choice is the logits'."""
    g = gen(3)
    for T, E in routes(6000):
        l = torch.randn(T, E, generator=g)
        l[::4] *= 100.0          # sigmoid: 1 and 0; softmax: below 2^-1000 of the largest
        l[1::4] += 45.0          # sigmoid: 1 - 1e-19
        l[2::4] -= 60.0          # sigmoid: 1e-26, lost in the bias
        bias = torch.full((E,), value)
        ref = l.sort(dim=1, descending=True, stable=True).indices[:, :6]
        for b in (bias.cuda(), None):
            r = moe.moe_router(l.cuda(), 6, routing=moe.RoutingParams(scoring, bias=b))
            assert torch.equal(r.ids.cpu().long(), ref), (T, E, b is None)
    for pair in ([40.0, 41.0], [-200.0, -199.0], [0.0, 1e-30]):
        r = moe.moe_router(torch.tensor([pair]).cuda(), 1, routing=moe.RoutingParams(scoring, bias=torch.full((2,), value).cuda()))
        assert r.ids.item() == 1


@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("value", [None, 0.0, 0.375])
def test_groups_of_scores_that_are_one(value, score):
    """Sigmoid scores from 37 on: a group's value is what its scores leave to 1, the smaller the better."""
    g = gen(4)
    for T, E in routes(6000):
        G, kept = 8, 3
        l = 38.0 + 20.0 * torch.rand(T, E, generator=g)
        bias = None if value is None else torch.full((E,), value).cuda()
        by = l.reshape(T, G, -1)
        top = by.sort(dim=2, descending=True).values[:, :, :1 if score == "max" else 2]
        rest = torch.exp(-top.double()).sum(2)   # 1 - sigmoid(l), to 1e-16 of itself
        order = rest.sort(dim=1, stable=True).indices[:, :kept]
        keep = torch.zeros(T, G, dtype=torch.bool).scatter_(1, order, True)
        ref = by.masked_fill(~keep[:, :, None], -math.inf).reshape(T, E).sort(dim=1, descending=True, stable=True).indices[:, :4]
        r = moe.moe_router(l.cuda(), 4, routing=moe.RoutingParams("sigmoid", n_group=G, topk_group=kept, bias=bias), group_score=score)
        assert torch.equal(r.ids.cpu().long(), ref), (T, E)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_scores_the_bias_swallows(scoring):
    """Scores of 1e-26 and less beside a bias of 1: the groups' order is that of the scores' sums."""
    g = gen(5)
    for T, E in routes(6000):
        G, kept = 8, 3
        l = -60.0 - 20.0 * torch.rand(T, E, generator=g)
        if scoring == "softmax":
            l[:, 0] = 0.0        # the largest score is 1, and its group the first
        by = l.reshape(T, G, -1)
        total = torch.exp(by.sort(dim=2, descending=True).values[:, :, :2].double()).sum(2)
        order = total.sort(dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros(T, G, dtype=torch.bool).scatter_(1, order, True)
        ref = by.masked_fill(~keep[:, :, None], -math.inf).reshape(T, E).sort(dim=1, descending=True, stable=True).indices[:, :4]
        r = moe.moe_router(l.cuda(), 4, routing=moe.RoutingParams(scoring, n_group=G, topk_group=kept, bias=torch.ones(E).cuda()))
        assert torch.equal(r.ids.cpu().long(), ref), (T, E)


# -------------------------------------------------------------------------------- scores that vanish
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,E", [(40, 64), (6000, 64), (6000, 100), (300, 250), (300, 1000)])
def test_tokens_whose_sigmoid_scores_vanish(T, E, dtype):
    """Their shares, the balance loss and its gradient are those of the formulas, whose scores are e^l there."""
    g = gen(6)
    l = torch.randn(T, E, generator=g) * 2
    l[::2] -= 75.0 + 400.0 * torch.rand(len(l[::2]), 1, generator=g)    # from 1e-33 to far below fp32's range
    l[1::6] -= 66.0                                                     # about where the shares change their form
    l[2, ::3], l[4, 1:], l[6] = -math.inf, -math.inf, -math.inf
    l = l.to(dtype)
    valid = torch.rand(T, generator=g) < 0.9
    valid[:8] = True
    dw = torch.randn(T, 4, generator=g)
    coef = 0.7 * T
    # in 64 bits, through logarithms
    x = l.double().requires_grad_()
    none = x.detach() == -math.inf
    live = valid & ~none.all(1)
    n = int(live.sum())
    safe = torch.where(live[:, None], torch.where(none, -1e5, x), 0.0)
    log = torch.nn.functional.logsigmoid(safe)
    share = torch.softmax(log, 1) * live[:, None]
    ids = torch.where(none, -math.inf, x.detach()).sort(dim=1, descending=True, stable=True).indices[:, :4]
    real = live[:, None] & ~none.gather(1, ids)
    counts = torch.bincount(ids[real], minlength=E)
    f = counts.double() * E / (4 * n)
    balance = (f * share.sum(0)).sum() / n
    w = torch.softmax(torch.where(real, log.gather(1, ids), torch.where(real.any(1, keepdim=True), -math.inf, 0.0)), 1) * real
    grad = torch.autograd.grad((w * dw.double()).sum() + coef * balance, x)[0].nan_to_num(0.0).detach()
    w, balance, share = w.detach(), balance.detach(), share.detach()

    r = moe.moe_router(l.cuda(), 4, routing=moe.RoutingParams("sigmoid"), valid=valid.cuda(), losses=True)
    assert torch.equal(r.ids.cpu().long(), torch.where(real, ids, -1))
    assert torch.equal(r.counts.cpu().long(), counts) and int(r.tokens) == n
    # fp32 half-steps: an exponential of a difference of up to 20 (the rest are below 2^-24 of the largest) 4 and 20, its sum 2 and
    # as many as a lane has experts, the quotient 4, twice; the sums over tokens
    u = 2 * (30 + E // 8) * 2.0 ** -24
    check_to = lambda got, want, size: ((got.double().cpu() - want).abs() <= size).all()  # noqa: E731
    assert check_to(r.weights, w, u * w + 1e-37)
    assert check_to(r.balance_loss, balance, (u + (T / 2432 + 80) * 2.0 ** -24) * balance)
    got = moe.moe_router_backward(l.cuda(), r, dw.cuda(), routing=moe.RoutingParams("sigmoid"), balance_coef=coef)
    h = coef * f / n
    size = share * (h + (share * h).sum(1, keepdim=True))
    inner = (w * dw.double().abs()).sum(1, keepdim=True)
    size = size.scatter_add(1, ids, torch.where(real, w * (dw.double().abs() + inner), 0.0))
    assert check_to(got, grad, torch.finfo(dtype).eps / 2 * grad.abs() + 4 * u * size + 1e-37)
    # what it was before: nothing of those tokens in the loss
    vanished = live & (l.double().max(1).values < -100)
    assert vanished.any() and abs(float(share[vanished].sum()) - int(vanished.sum())) < 1e-6


# ------------------------------------------------------ tokens that four to a warp leave to the whole warp
SHARED = [base.Case(6000, E, k, scoring, bias, groups, kept, score, renorm, 1.5, dtype, padding)
          for E, k, scoring, bias, groups, kept, score, renorm, dtype, padding in (
    (64, 15, "softmax", "steps", 1, 1, "top2", True, torch.float32, 0.1),
    (64, 16, "softmax", "", 1, 1, "top2", False, torch.bfloat16, 0.0),
    (64, 16, "sigmoid", "steps", 1, 1, "top2", True, torch.float32, 0.2),
    (64, 17, "sigmoid", "", 1, 1, "top2", True, torch.float16, 0.0),
    (64, 32, "softmax", "steps", 1, 1, "top2", False, torch.float32, 0.3),
    (64, 15, "sigmoid", "large", 8, 4, "top2", True, torch.float32, 0.0),
    (64, 16, "softmax", "zero", 8, 3, "max", True, torch.float32, 0.1),
    (128, 15, "sigmoid", "steps", 8, 2, "top2", False, torch.bfloat16, 0.0),
    (128, 16, "sigmoid", "steps", 4, 2, "max", True, torch.float32, 0.1),
    (128, 17, "softmax", "", 2, 1, "top2", True, torch.float32, 0.0),
    (128, 32, "sigmoid", "large", 8, 3, "top2", True, torch.float32, 0.1),
    (100, 32, "softmax", "", 5, 4, "top2", False, torch.float16, 0.5))]


@pytest.mark.parametrize("c", SHARED, ids=str)
def test_many_choices_of_many_tokens(c):
    base.test_choice_weights_and_loads(c)


@pytest.mark.parametrize("c", SHARED[::3], ids=str)
def test_gradient_of_many_choices(c):
    base.test_gradient(c, True)


@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_keys_closer_than_their_fp32_error_of_many_tokens(scoring, groups, kept):
    g = gen(7)
    for E in (64, 128):
        l = torch.randn(1, E, generator=g) + torch.randn(6000, E, generator=g) * 1e-7
        s = score64(l[:1], scoring)[0]
        bias = (1.0 - s).float()
        c = base.Case(6000, E, 8, scoring, "given", groups, kept)
        r = moe.moe_router(l.cuda(), 8, routing=base.routing(c, bias.cuda()))
        assert torch.equal(r.ids.cpu().long(), base.reference(c, l, bias, None)["ids"])


@pytest.mark.parametrize("T", [5, 6000])
def test_all_equal_keys_of_many_tokens(T):
    for scoring in ("softmax", "sigmoid"):
        for bias in (None, torch.full((64,), 0.25, device="cuda")):
            for dtype in (torch.float32, torch.bfloat16):
                x = torch.zeros(T, 64, dtype=dtype, device="cuda")
                for groups, kept, k in ((1, 1, 6), (8, 2, 10), (1, 1, 32)):
                    rp = moe.RoutingParams(scoring, n_group=groups, topk_group=kept, bias=bias)
                    r = moe.moe_router(x, k, routing=rp, losses=True)
                    assert torch.equal(r.ids.cpu(), torch.arange(k, dtype=torch.int32).expand(T, k))
                    assert torch.allclose(r.weights, torch.full_like(r.weights, 1 / k), rtol=1e-6)
                    assert r.counts.tolist() == [T] * k + [0] * (64 - k)


@pytest.mark.parametrize("score", ["top2", "max"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [40, 6000])
def test_masked_experts_in_groups_keep_their_shares(T, scoring, score):
    """A bias of -inf takes an expert out of the choice and its group's value; the scores of the others are the same as before, and
    it keeps its share in the balance loss."""
    g = gen(8)
    for E, groups, kept in ((64, 8, 3), (60, 6, 2), (128, 4, 2)):
        l = torch.randn(T, E, generator=g)
        bias = torch.randint(-40, 41, (E,), generator=g) * 0.001
        gone = torch.zeros(E, dtype=torch.bool)
        gone[::3] = True
        gone[:E // groups - 1] = True        # all but one of the first group
        gone[-(E // groups):] = True         # all of the last
        bias[gone] = -math.inf
        s = score64(l, scoring)
        key = s + bias.double()
        top = key.reshape(T, groups, -1).sort(dim=2, descending=True).values[:, :, :1 if score == "max" else 2]
        none = (top == -math.inf).all(2)
        value = torch.where(top == -math.inf, 0.0, top).sum(2).masked_fill(none, -math.inf)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, order, True).repeat_interleave(E // groups, 1)
        best = key.masked_fill(~keep, -math.inf).sort(dim=1, descending=True, stable=True)
        ids = torch.where(best.values > -math.inf, best.indices, -1)[:, :4]
        rp = moe.RoutingParams(scoring, n_group=groups, topk_group=kept, bias=bias.cuda())
        r = moe.moe_router(l.cuda(), 4, routing=rp, group_score=score, losses=True)
        assert torch.equal(r.ids.cpu().long(), ids)
        counts = torch.bincount(ids[ids >= 0], minlength=E)
        assert torch.equal(r.counts.cpu().long(), counts) and int(r.tokens) == T
        want = (counts.double() * E / (4 * T) * (s / s.sum(1, keepdim=True)).mean(0)).sum()
        # a score and its sum: 4 half-steps each, the argument's rounding (|l| < 8), the lane's and the tokens' sums
        assert abs(float(r.balance_loss) - float(want)) <= (40 + E // 8 + T / 2432 + 80) * 2.0 ** -24 * float(want)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_values_pass_fp32(scoring, sign):
    """Sums of two keys with finite biases near fp32's largest number: the larger sum, and at equal ones the scores' sum."""
    g = gen(9)
    for T, E in routes(6000):
        G, kept, size = 8, 3, E // 8
        l = torch.randn(T, E, generator=g)
        level = torch.tensor([3.0, 2.0, 3.0, 2.5, 3.0, 2.0, 3.0, 3.0]) * sign * 1e38
        bias = level.repeat_interleave(size)
        s = score64(l, scoring).reshape(T, G, size).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        # by the level, then the scores (a group's own two best keys are equal in fp64: by their logits, so by their scores)
        rank = torch.unique(level, sorted=True, return_inverse=True)[1]
        order = (rank.double() * 10 + s).sort(dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros(T, G, dtype=torch.bool).scatter_(1, order, True).repeat_interleave(size, 1)
        key = (rank.double().repeat_interleave(size) * 1000 + l.double()).masked_fill(~keep, -math.inf)
        ids = key.sort(dim=1, descending=True, stable=True).indices[:, :4]
        rp = moe.RoutingParams(scoring, n_group=G, topk_group=kept, bias=bias.cuda())
        r = moe.moe_router(l.cuda(), 4, routing=rp)
        assert torch.equal(r.ids.cpu().long(), ids), (T, E)
