"""The norms before and after a block, and their gradients, against 64-bit values."""
import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from train_testutil import DTYPES, check, gen, ids_of, offset_copy, rand, strided_copy

pytestmark = pytest.mark.gpu

# fp32 roundings of one value beyond the rounding to its type: a row's sum of squares is summed by at
# most 32 terms per thread, 5 lane steps and 16 warps (53, halved by the square root), the root, the mean
# and five products; a row's dot product 53 more
ROW = 53 / 2 + 8
SHAPES = [(1, 1), (1, 7168), (3, 8), (5, 33), (64, 256), (7, 1000), (301, 520), (2, 16384), (3, 16383), (400, 2880),
          (160, 4104), (19, 4097), (1000, 64), (2100, 1032), (700, 7168), (310, 16384), (320, 8448)]


def norm64(x, w, off, eps):
    x = x.double().cpu()
    r = 1 / torch.sqrt((x * x).mean(1) + eps)
    return x * r[:, None] * (w.double().cpu() + off), r


def gate64(gate, kind, sigmoid):
    if kind == "none":
        return torch.ones(1, 1, dtype=torch.float64)
    g = gate.double().cpu()
    g = torch.sigmoid(g) if sigmoid else g
    return g.reshape(-1, 1) if kind == "token" else g.reshape(1, -1) if kind == "channel" else g


def make_gate(g, kind, T, H, dtype):
    shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[kind]
    return None if shape is None else rand(g, *shape, dtype=dtype)


@pytest.mark.parametrize("wtype", ["fp32", "same"])
@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,H", SHAPES)
def test_pre_norm_and_gradient(T, H, dtype, wtype):
    g = gen(T * 7 + H)
    wt = torch.float32 if wtype == "fp32" else dtype
    off = 1.0 if wtype == "same" else 0.0
    x, w = rand(g, T, H, dtype=dtype), rand(g, H, dtype=wt, std=0.2) + (1 - off)
    h, rstd = moe.moe_pre_norm(x, w, eps=1e-5, weight_offset=off)
    want, r = norm64(x, w, off, 1e-5)
    check(h, want, roundings=ROW, name="h")
    check(rstd, r, roundings=ROW, name="rstd")
    dh, dres = rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype)
    for res in (dres, None):
        dx, dw = moe.moe_pre_norm_backward(dh, x, w, rstd, dresidual=res, weight_offset=off)
        rs, xx, dd = rstd.double().cpu()[:, None], x.double().cpu(), dh.double().cpu()
        t, n = dd * (w.double().cpu() + off), xx * rs
        rr = 0 if res is None else res.double().cpu()
        m = (t * n).mean(1, keepdim=True)
        ma = (t * n).abs().mean(1, keepdim=True)
        size = rs * (t.abs() + n.abs() * ma) + (0 if res is None else rr.abs())
        check(dx, rs * (t - n * m) + rr, size, 53 + 8, "dx")
        # rows are summed by one CTA after another, its groups and the CTAs joined: at most T + 40 additions
        check(dw, (dd * n).sum(0), (dd * n).abs().sum(0), T + 44, "dweight")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("kind", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7168), (5, 33), (64, 256), (301, 520), (2, 16384), (3, 16383), (400, 2880),
                                 (19, 4097), (2100, 1032), (700, 7168), (310, 16384), (320, 8448)])
def test_post_norm_and_gradient(T, H, dtype, kind, sigmoid):
    if kind == "none" and sigmoid:
        pytest.skip("no gate to take the sigmoid of")
    g = gen(T + 3 * H)
    a, b, eps, off = 0.75, 0.3, 1e-6, 0.5
    y, res, gate = rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype), make_gate(g, kind, T, H, dtype)
    w, w2 = rand(g, H, dtype=dtype), rand(g, H, dtype=dtype)
    kw = dict(gate=gate, gate_kind=kind, gate_sigmoid=sigmoid, residual_scale=a, block_scale=b, weight_offset=off)
    p = moe.moe_post_norm(y, res, w, eps=eps, **kw)
    z, r = norm64(y, w, off, eps)
    G = gate64(gate, kind, sigmoid)
    out = a * res.double().cpu() + b * G * z
    size = (a * res.double().cpu()).abs() + (b * G * z).abs()
    check(p.out, out, size, ROW + 12, "out")       # 12: the sigmoid's and the scales' roundings
    check(p.rstd, r, roundings=ROW, name="rstd")
    assert p.next_h is None and p.next_rstd is None
    q = moe.moe_post_norm(y, res, w, eps=eps, next_weight=w2, **kw)
    assert torch.equal(q.out, p.out) and torch.equal(q.rstd, p.rstd)
    h2, r2 = norm64(p.out, w2, off, eps)
    check(q.next_h, h2, roundings=ROW, name="next_h")
    check(q.next_rstd, r2, roundings=ROW, name="next_rstd")

    dout = rand(g, T, H, dtype=dtype)
    d = moe.moe_post_norm_backward(dout, y, w, p.rstd, **kw)
    rs, n, dd = p.rstd.double().cpu()[:, None], y.double().cpu() * p.rstd.double().cpu()[:, None], dout.double().cpu()
    ww = w.double().cpu() + off
    t = b * G * dd * ww
    m, ma = (t * n).mean(1, keepdim=True), (t * n).abs().mean(1, keepdim=True)
    check(d.dy, rs * (t - n * m), rs * (t.abs() + n.abs() * ma), 53 + 20, "dy")
    check(d.dresidual, a * dd, roundings=1, name="dresidual")
    s = b * G * dd * n
    check(d.dweight, s.sum(0), s.abs().sum(0), T + 60, "dweight")
    if kind == "none":
        assert d.dgate is None
    else:
        # (1 - sigmoid cancels where the sigmoid is near one: its error there is a rounding of the sigmoid)
        slope = G * (1 - G) if sigmoid else torch.ones_like(G)
        loose = G if sigmoid else torch.ones_like(G)
        s, size = slope * b * dd * n * ww, (loose * b * dd * n * ww).abs()
        if kind == "token":
            check(d.dgate, s.sum(1), size.sum(1), 53 + 20, "dgate")
        elif kind == "channel":
            assert d.dgate.dtype == torch.float32
            check(d.dgate, s.sum(0), size.sum(0), T + 60, "dgate")
        else:
            check(d.dgate, s, size, 20, "dgate")
    e = moe.moe_post_norm_backward(dout, y, w, p.rstd, residual_grad=False, **kw)
    assert e.dresidual is None and torch.equal(e.dy, d.dy) and torch.equal(e.dweight, d.dweight)


@pytest.mark.parametrize("kind,sigmoid", [("none", False), ("token", True), ("channel", True), ("full", True),
                                          ("full", False)])
def test_gradients_against_differences(kind, sigmoid):
    """The kernels' gradients in fp32 along a random direction against central differences of the
    formula in 64 bits (step 1e-5: differences good to about 1e-9)."""
    g = gen(17)
    T, H, a, b, eps = 9, 72, 0.9, 0.4, 1e-6
    x, y, w = rand(g, T, H), rand(g, T, H), rand(g, H)
    gate = make_gate(g, kind, T, H, torch.float32)
    dout, dh = rand(g, T, H), rand(g, T, H)
    vy, vw, vx = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((T, H), (H,), (T, H)))
    vg = None if gate is None else torch.randn(gate.shape, generator=g, dtype=torch.float64)
    y64, w64, x64 = y.double().cpu(), w.double().cpu(), x.double().cpu()
    g64 = None if gate is None else gate.double().cpu()

    def loss(s):
        z, _ = norm64(y64 + s * vy, w64 + s * vw, 0, eps)
        gg = gate64(None if gate is None else g64 + s * vg, kind, sigmoid)
        out = a * (x64 + s * vx) + b * gg * z
        h, _ = norm64(x64 + s * vx, w64 + s * vw, 0, eps)
        return ((out * dout.double().cpu()).sum() + (h * dh.double().cpu()).sum()).item()
    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    _, rx = moe.moe_pre_norm(x, w, eps=eps)
    kw = dict(gate=gate, gate_kind=kind, gate_sigmoid=sigmoid, residual_scale=a, block_scale=b)
    p = moe.moe_post_norm(y, x, w, eps=eps, **kw)
    d = moe.moe_post_norm_backward(dout, y, w, p.rstd, **kw)
    dx, dw = moe.moe_pre_norm_backward(dh, x, w, rx, dresidual=d.dresidual)
    terms = [(d.dy, vy), (dx, vx), (dw + d.dweight, vw)] + ([] if gate is None else [(d.dgate, vg)])
    got = sum((u.double().cpu() * v.reshape(u.shape)).sum().item() for u, v in terms)
    mass = sum((u.double().cpu() * v.reshape(u.shape)).abs().sum().item() for u, v in terms)
    assert abs(got - want) <= 1e-5 * mass


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
def test_layouts(dtype):
    """Odd addresses, rows inside wider matrices, a gate column of a wider matrix: the same values."""
    g = gen(23)
    for T, H in ((33, 264), (12, 97)):
        x, y, d, w = rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype), rand(g, H)
        gt, gf = rand(g, T, dtype=dtype), rand(g, T, H, dtype=dtype)
        for lay in (offset_copy, lambda t: strided_copy(t, 7, 3), lambda t: strided_copy(t, 64, 32)):
            want, r = norm64(x, w, 0, 1e-6)
            h, rstd = moe.moe_pre_norm(lay(x), offset_copy(w))
            check(h, want, roundings=ROW, name="h")
            check(rstd, r, roundings=ROW, name="rstd")
            col = strided_copy(gt[:, None].expand(T, 3).contiguous(), 2)[:, 1:2]
            p = moe.moe_post_norm(lay(y), lay(x), w, gate=col, gate_kind="token", next_weight=w)
            z = gt.double().cpu()[:, None] * norm64(y, w, 0, 1e-6)[0]
            check(p.out, x.double().cpu() + z, x.double().cpu().abs() + z.abs(), ROW + 4, "out")
            check(p.next_h, norm64(p.out, w, 0, 1e-6)[0], roundings=ROW, name="next_h")
            f = moe.moe_post_norm_backward(lay(d), lay(y), w, rstd, gate=lay(gf), gate_kind="full", gate_sigmoid=True)
            f0 = moe.moe_post_norm_backward(d, y, w, rstd, gate=gf, gate_kind="full", gate_sigmoid=True)
            for u, v in ((f.dgate, f0.dgate), (f.dresidual, f0.dresidual)):
                assert torch.equal(u, v)
            k = moe.moe_post_norm_backward(lay(d), lay(y), w, rstd, gate=col, gate_kind="token")
            assert k.dgate.shape == (T, 1)
            n = y.double().cpu() * rstd.double().cpu()[:, None]
            s = d.double().cpu() * n * w.double().cpu()
            check(k.dgate, s.sum(1, keepdim=True), s.abs().sum(1, keepdim=True), 80, "dgate")


def test_rows_of_zeros_infinities_and_nan():
    w = torch.ones(64, device="cuda")
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    x[1, 3], x[2, 5], x[3] = float("inf"), float("nan"), 1
    h, rstd = moe.moe_pre_norm(x, w, eps=1e-6)
    assert torch.equal(h[0], torch.zeros_like(h[0])) and abs(rstd[0].item() - 1e3) < 1e-3
    assert torch.isnan(h[1, 3]) and h[1, 0].item() == 0 and torch.isnan(h[2]).all()
    assert torch.equal(h[3], torch.ones_like(h[3]))
    dx, dw = moe.moe_pre_norm_backward(x[[0, 3]], x[[0, 3]], w, rstd[[0, 3]].contiguous())
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_no_rows():
    x, w = torch.zeros(0, 96, device="cuda"), torch.ones(96, device="cuda")
    h, rstd = moe.moe_pre_norm(x, w)
    assert h.shape == (0, 96) and rstd.shape == (0,)
    dx, dw = moe.moe_pre_norm_backward(x, x, w, rstd)
    assert dx.shape == (0, 96) and torch.equal(dw, torch.zeros(96, device="cuda"))
    p = moe.moe_post_norm(x, x, w, gate=w, gate_kind="channel", next_weight=w)
    assert p.out.shape == (0, 96)
    d = moe.moe_post_norm_backward(x, x, w, rstd, gate=w, gate_kind="channel")
    assert torch.equal(d.dweight, torch.zeros(96, device="cuda")) and torch.equal(d.dgate, d.dweight)


def test_repeats_stream_and_graph():
    """The same bits every time (no atomics), on another stream and from a graph with new inputs."""
    g = gen(29)
    T, H = 333, 1032
    x, y, d = (rand(g, T, H, dtype=torch.bfloat16) for _ in range(3))
    w, gate = rand(g, H), rand(g, T, dtype=torch.bfloat16)

    def step():
        h, r = moe.moe_pre_norm(x, w)
        p = moe.moe_post_norm(y, x, w, gate=gate, gate_kind="token", gate_sigmoid=True, next_weight=w)
        b = moe.moe_post_norm_backward(d, y, w, p.rstd, gate=gate, gate_kind="token", gate_sigmoid=True)
        dx, dw = moe.moe_pre_norm_backward(d, x, w, r, dresidual=b.dresidual)
        return h, p.out, p.next_h, b.dy, b.dweight, b.dgate, dx, dw
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for t in (x, y, d):
        t.copy_(rand(g, T, H, dtype=torch.bfloat16))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,H", [(40, 1), (40, 7), (60, 249), (60, 250), (40, 1753), (200, 4811), (30, 9001)])
def test_rows_between_sixteen_byte_boundaries(T, H, dtype):
    """Rows that share 16 bytes with their neighbours."""
    test_pre_norm_and_gradient(T, H, dtype, "same")
    for kind, sigmoid in (("token", False), ("channel", True), ("full", False), ("full", True)):
        test_post_norm_and_gradient(T, H, dtype, kind, sigmoid)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
def test_neighbours_that_are_not_finite(dtype):
    g = gen(5)
    T, H = 40, 251
    x, w, d = rand(g, T, H, dtype=dtype), rand(g, H), rand(g, T, H, dtype=dtype)
    x[20] = float("nan")
    x[22, 3] = float("inf")
    h, rstd = moe.moe_pre_norm(x, w, eps=1e-5)
    want, _ = norm64(x, w, 0, 1e-5)
    keep = [t for t in range(T) if t not in (20, 22)]
    check(h[keep], want[keep], roundings=ROW, name="h")
    assert h[20].isnan().all()
    p = moe.moe_post_norm(x, d, w, eps=1e-5, next_weight=w)
    assert torch.isfinite(p.next_h[keep]).all() and torch.isfinite(p.out[keep]).all()
    dx, _ = moe.moe_pre_norm_backward(d, x, w, rstd)
    assert torch.isfinite(dx[keep]).all() and dx[20].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,H", [(310, 1), (311, 3), (333, 249), (2101, 250), (700, 1753), (400, 4811), (320, 9001)])
def test_many_rows_between_sixteen_byte_boundaries(T, H, dtype):
    """Enough rows for the ring, whose rows start by their number modulo 8."""
    test_pre_norm_and_gradient(T, H, dtype, "fp32")
    for kind, sigmoid in (("none", False), ("token", True), ("channel", True), ("full", False), ("full", True)):
        test_post_norm_and_gradient(T, H, dtype, kind, sigmoid)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("pad,lead", [(16, 0), (16, 8), (7, 3)])
def test_many_strided_rows_and_their_neighbours(pad, lead, dtype):
    """Rows of wider matrices (NaN between them), some of them not finite: the others are as without."""
    g = gen(pad + lead)
    T, H = 330, 251
    lay = lambda t: strided_copy(t, pad, lead)
    x, w, d = rand(g, T, H, dtype=dtype), rand(g, H), rand(g, T, H, dtype=dtype)
    x[100], x[329], x[200, 7] = float("nan"), float("nan"), float("inf")
    keep = torch.tensor([t for t in range(T) if t not in (100, 200, 329)])
    h, rstd = moe.moe_pre_norm(lay(x), w, eps=1e-5)
    want, _ = norm64(x, w, 0, 1e-5)
    check(h.cpu()[keep], want[keep], roundings=ROW, name="h")
    assert h[100].isnan().all() and h[329].isnan().all()
    p = moe.moe_post_norm(lay(x), lay(d), w, eps=1e-5, next_weight=w)
    z = d.double().cpu() + want
    check(p.out.cpu()[keep], z[keep], (d.double().cpu().abs() + want.abs())[keep], ROW + 12, "out")
    check(p.next_h.cpu()[keep], norm64(p.out, w, 0, 1e-5)[0][keep], roundings=ROW, name="next_h")
    dx, _ = moe.moe_pre_norm_backward(lay(d), lay(x), w, rstd, dresidual=lay(d))
    assert torch.isfinite(dx.cpu()[keep]).all() and dx[100].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,H", [(1, 9001), (5, 8193), (7, 12001), (100, 16381), (303, 10003), (304, 8199)])
def test_few_wide_rows_between_sixteen_byte_boundaries(T, H, dtype):
    test_pre_norm_and_gradient(T, H, dtype, "fp32")
    for kind, sigmoid in (("none", False), ("full", True)):
        test_post_norm_and_gradient(T, H, dtype, kind, sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("kind", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
def test_no_rows_with_each_gate(kind, sigmoid, dtype):
    H = 96
    x, w = torch.zeros(0, H, device="cuda", dtype=dtype), torch.ones(H, device="cuda")
    gate = make_gate(gen(1), kind, 0, H, dtype)
    kw = dict(gate=gate, gate_kind=kind, gate_sigmoid=sigmoid and kind != "none")
    p = moe.moe_post_norm(x, x, w, next_weight=w, **kw)
    assert p.out.shape == p.next_h.shape == (0, H) and p.rstd.shape == p.next_rstd.shape == (0,)
    torch.full((H,), float("nan"), device="cuda")   # memory that the sums take next
    d = moe.moe_post_norm_backward(x, x, w, p.rstd, **kw)
    assert d.dy.shape == d.dresidual.shape == (0, H) and torch.equal(d.dweight, torch.zeros(H, device="cuda"))
    assert (d.dgate is None) == (kind == "none")
    if kind == "channel":
        assert torch.equal(d.dgate, torch.zeros(H, device="cuda"))
    elif gate is not None:
        assert d.dgate.shape == gate.shape and d.dgate.dtype == dtype


@pytest.mark.parametrize("kind", ["token", "channel", "full"])
@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,H", [(1, 8), (7, 264), (40, 97), (700, 1032), (333, 249)])
def test_gradients_of_saturated_gates(T, H, dtype, kind):
    """Gates from -30 to 30, where s * (1 - s) of a rounded sigmoid s has no digits left: errors count against the
    slope itself, d/dg sigmoid = e / (1 + e)^2 with e = exp(-|g|).  An fp32 exponential of an argument |g| is off
    by at most 2 |g| + 4 half-steps, the quotient and the products by 12 more."""
    g = gen(T + H)
    b = 1024.0   # the slopes in fp16's normal range
    y, dout, w = rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype), rand(g, H)
    gate = make_gate(g, kind, T, H, dtype)
    big = torch.tensor([8.0, -8, 10, -10, 12, -12, 16, -16, 17, -17, 20, -20, 30, -30], dtype=dtype, device="cuda")
    gate.view(-1).copy_(big[torch.arange(gate.numel(), device="cuda") % len(big)])
    rstd = norm64(y, w, 0, 1e-6)[1].float().cuda()
    d = moe.moe_post_norm_backward(dout, y, w, rstd, gate=gate, gate_kind=kind, gate_sigmoid=True, block_scale=b)
    g64 = gate.double().cpu()
    g64 = g64.reshape(-1, 1) if kind == "token" else g64.reshape(1, -1) if kind == "channel" else g64
    e = torch.exp(-g64.abs())
    slope, sig = e / (1 + e) ** 2, torch.where(g64 < 0, e, torch.ones_like(e)) / (1 + e)
    n, dd, ww = y.double().cpu() * rstd.double().cpu()[:, None], dout.double().cpu(), w.double().cpu()
    s = slope * b * dd * n * ww
    exp_error = 2 * 30 + 4 + 12
    if kind == "full":
        check(d.dgate, s, roundings=exp_error, name="dgate")
    else:
        check(d.dgate, s.sum(0 if kind == "channel" else 1), s.abs().sum(0 if kind == "channel" else 1),
              exp_error + (T + 60 if kind == "channel" else 53 + 20), "dgate")
    t = b * sig * dd * ww
    m, ma = (t * n).mean(1, keepdim=True), (t * n).abs().mean(1, keepdim=True)
    rs = rstd.double().cpu()[:, None]
    check(d.dy, rs * (t - n * m), rs * (t.abs() + n.abs() * ma), exp_error + 53 + 20, "dy")
    s = b * sig * dd * n
    check(d.dweight, s.sum(0), s.abs().sum(0), exp_error + T + 60, "dweight")


def test_rows_past_two_to_the_31_elements():
    """Row offsets that pass 32 bits: the last rows equal the same rows in a matrix of their own."""
    T, H = 264000, 8200
    g = torch.Generator(device="cuda").manual_seed(3)
    some = [torch.randn(64, H, generator=g, device="cuda").bfloat16() for _ in range(3)]
    x, y, gate = (s.repeat(T // 64, 1) for s in some)
    w = torch.randn(H, generator=g, device="cuda")
    kw = dict(gate_kind="full", gate_sigmoid=True, block_scale=0.5)
    h, rstd = moe.moe_pre_norm(x, w)
    h1, rstd1 = moe.moe_pre_norm(some[0].repeat(10, 1), w)
    for at in (slice(0, 640), slice(T - 640, T)):
        assert torch.equal(h[at], h1) and torch.equal(rstd[at], rstd1)
    del h
    p = moe.moe_post_norm(y, x, w, gate=gate, next_weight=w, **kw)
    p1 = moe.moe_post_norm(some[1].repeat(10, 1), some[0].repeat(10, 1), w, gate=some[2].repeat(10, 1), next_weight=w, **kw)
    for at in (slice(0, 640), slice(T - 640, T)):
        assert torch.equal(p.out[at], p1.out) and torch.equal(p.next_h[at], p1.next_h)
    del p.out, p.next_h
    d = moe.moe_post_norm_backward(x, y, w, p.rstd, gate=gate, **kw)
    d1 = moe.moe_post_norm_backward(some[0].repeat(10, 1), some[1].repeat(10, 1), w, p1.rstd, gate=some[2].repeat(10, 1),
                                    **kw)
    dx, _ = moe.moe_pre_norm_backward(d.dresidual, x, w, rstd, dresidual=d.dy)
    dx1, _ = moe.moe_pre_norm_backward(d1.dresidual, some[0].repeat(10, 1), w, rstd1, dresidual=d1.dy)
    for at in (slice(0, 640), slice(T - 640, T)):
        for a, b in ((d.dy, d1.dy), (d.dresidual, d1.dresidual), (d.dgate, d1.dgate), (dx, dx1)):
            assert torch.equal(a[at], b)
