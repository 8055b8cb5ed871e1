"""The training router's masks and borders: experts masked by their bias, keys that meet in 64 bits, scores that vanish, and the same
decisions where four tokens share a warp."""
import math

import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
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
