"""Token rows sorted by expert and back, and their gradients, against 64-bit values on the CPU."""
import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from train_testutil import (DTYPES, check, gen, ids_of, offset_copy, rand, status, status_clear, strided_copy)

pytestmark = pytest.mark.gpu


def make_ids(g, T, k, E, drop=0.0, skew=False):
    """Expert ids; with drop, some are -1 and (T > 2) token 1 has none left."""
    if skew:
        ids = (torch.rand(T, k, generator=g) ** 3 * E).long().clamp(max=E - 1)
    else:
        ids = torch.randint(0, E, (T, k), generator=g)
    if drop:
        ids[torch.rand(T, k, generator=g) < drop] = -1
        if T > 2:
            ids[1] = -1
    return ids.int()


def sort_ref(ids, E):
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(p)
    offsets, order = [0], []
    for one in lists:
        order += one
        offsets.append(len(order))
    pos = [-1] * len(flat)
    for r, p in enumerate(order):
        pos[p] = r
    return (torch.tensor(offsets), torch.tensor(order + [-1] * (len(flat) - len(order))),
            torch.tensor(pos).reshape(ids.shape))


def check_dispatch(d, x, ids, E):
    offsets, pair_ids, pos = sort_ref(ids.cpu(), E)
    assert torch.equal(d.expert_offsets.cpu().long(), offsets)
    assert torch.equal(d.pair_ids.cpu().long(), pair_ids)
    assert torch.equal(d.pos.cpu().long(), pos)
    k = ids.shape[1]
    want = torch.zeros(ids.numel(), x.shape[1], dtype=x.dtype)
    n = int(offsets[-1])
    want[:n] = x.cpu()[pair_ids[:n] // k]
    assert torch.equal(d.rows.cpu(), want)


CASES = [  # T, k, E, H, drop, skew
    (1, 1, 1, 1, 0.0, False),
    (1, 8, 256, 7168, 0.0, False),
    (2, 3, 5, 3, 0.5, False),
    (7, 2, 4, 100, 0.3, False),
    (33, 32, 1024, 24, 0.1, True),
    (64, 8, 128, 520, 0.0, True),
    (300, 6, 33, 136, 0.05, True),
    (1025, 1, 7, 65, 0.0, True),
    (2049, 8, 257, 40, 0.02, False),      # more pairs than one launch counts
    (5000, 7, 1024, 9, 0.02, True),
    (9001, 4, 3, 16, 0.0, True),
    (700, 3, 16, 7168, 0.1, False),       # rows in several pieces; many slabs of columns
    (3000, 8, 1024, 1032, 0.1, True),
    (1500, 20, 64, 264, 0.05, True),
    (400, 32, 40, 4096, 0.3, False),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,k,E,H,drop,skew", CASES)
def test_dispatch(T, k, E, H, drop, skew, dtype):
    g = gen(T + k)
    ids = make_ids(g, T, k, E, drop, skew).cuda()
    x = rand(g, T, H, dtype=dtype)
    status_clear()
    check_dispatch(moe.moe_dispatch(x, ids, E), x, ids, E)
    assert status() == 0


@pytest.mark.parametrize("pairs", [16383, 16384, 16385, 152 * 1024 + 1])
def test_dispatch_at_the_counting_limit(pairs):
    g = gen(pairs)
    ids = make_ids(g, pairs, 1, 61, 0.01).cuda()
    x = rand(g, pairs, 8, dtype=torch.bfloat16)
    check_dispatch(moe.moe_dispatch(x, ids, 61), x, ids, 61)


def test_dispatch_without_tokens_or_experts_left():
    x = torch.zeros(0, 16, device="cuda", dtype=torch.bfloat16)
    d = moe.moe_dispatch(x, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert d.rows.shape == (0, 16) and d.expert_offsets.tolist() == [0] * 10
    assert moe.moe_combine(d.rows, d.pos).shape == (0, 16)
    x = torch.ones(40, 16, device="cuda")
    d = moe.moe_dispatch(x, torch.full((40, 3), -1, dtype=torch.int32, device="cuda"), 9)
    assert d.expert_offsets.tolist() == [0] * 10 and d.rows.abs().sum().item() == 0
    assert torch.all(d.pos == -1) and torch.all(d.pair_ids == -1)
    y = torch.full((120, 16), float("nan"), device="cuda")    # rows of no pair are not read
    assert torch.equal(moe.moe_combine(y, d.pos), torch.zeros(40, 16, device="cuda"))
    dy, dw = moe.moe_combine_backward(x, y, d.pos, d.pair_ids, torch.ones(40, 3, device="cuda"))
    assert dy.abs().sum().item() == 0 and dw.abs().sum().item() == 0


def test_dispatch_reports_ids_past_the_experts():
    g = gen(3)
    ids = make_ids(g, 50, 4, 12)
    ids[3, 1], ids[49, 3] = 12, 2 ** 31 - 1
    ids = ids.cuda()
    x = rand(g, 50, 32)
    status_clear()
    check_dispatch(moe.moe_dispatch(x, ids, 12), x, ids, 12)
    assert status() == 2
    ids = torch.randint(0, 5, (20000, 1), generator=g, dtype=torch.int32).cuda()
    ids[777] = 5
    x = rand(g, 20000, 4)
    check_dispatch(moe.moe_dispatch(x, ids, 5), x, ids, 5)
    assert status() == 2


@pytest.mark.parametrize("layout", ["offset", "strided", "strided_wide"])
@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
def test_layouts(layout, dtype):
    """Rows at odd addresses, inside wider matrices, and of every vector width."""
    g = gen(11)
    lay = {"offset": offset_copy, "strided": lambda t: strided_copy(t, 5, 2),
           "strided_wide": lambda t: strided_copy(t, 64, 32)}[layout]
    for H in (24, 25, 26, 28):
        T, k, E = 37, 4, 6
        ids = make_ids(g, T, k, E, 0.1).cuda()
        x, w = rand(g, T, H, dtype=dtype), rand(g, T, k)
        d = moe.moe_dispatch(lay(x), ids, E)
        check_dispatch(d, x, ids, E)
        y, dout = rand(g, T * k, H, dtype=dtype), rand(g, T, H, dtype=dtype)
        assert torch.equal(moe.moe_combine(lay(y), d.pos, w), moe.moe_combine(y, d.pos, w))
        assert torch.equal(moe.moe_dispatch_backward(lay(y), d.pos), moe.moe_dispatch_backward(y, d.pos))
        a, b = moe.moe_combine_backward(lay(dout), lay(y), d.pos, d.pair_ids, w)
        dy, dw = combine_backward_ref(dout, y, d.pos, w)
        check(a, dy, name="dy")
        check(b, dw[0], dw[1], H, "dweights")


def combine_ref(y, pos, w):
    """(sum, sum of magnitudes) in 64 bits."""
    y, pos = y.cpu().double(), pos.cpu().long()
    T, k = pos.shape
    out, size = torch.zeros(T, y.shape[1], dtype=torch.float64), torch.zeros(T, y.shape[1], dtype=torch.float64)
    for j in range(k):
        live = pos[:, j] >= 0
        term = y[pos[live, j]] * (1.0 if w is None else w.cpu().double()[live, j:j + 1])
        out[live] += term
        size[live] += term.abs()
    return out, size


def combine_backward_ref(dout, y, pos, w):
    dout, y, pos, w = dout.cpu().double(), y.cpu().double(), pos.cpu().long(), w.cpu().double()
    T, k = pos.shape
    dy, dw, size = torch.zeros_like(y), torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0).reshape(-1)
        dy[pos[t, j]] = w[t, j:j + 1] * dout[t]
        dw[t, j] = (dout[t] * y[pos[t, j]]).sum(1)
        size[t, j] = (dout[t] * y[pos[t, j]]).abs().sum(1)
    return dy, (dw, size)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,k,E,H,drop,skew", CASES)
def test_combine_and_gradients(T, k, E, H, drop, skew, dtype):
    g = gen(T + H)
    ids = make_ids(g, T, k, E, drop, skew)
    _, pair_ids, pos = sort_ref(ids, E)
    pos, pair_ids = pos.int().cuda(), pair_ids.int().cuda()
    y, w, dout = rand(g, T * k, H, dtype=dtype), rand(g, T, k), rand(g, T, H, dtype=dtype)
    for weights in (w, None):
        out, size = combine_ref(y, pos, weights)
        check(moe.moe_combine(y, pos, weights), out, size, k + 1, "out")
    out, size = combine_ref(y, pos, None)
    check(moe.moe_dispatch_backward(y, pos), out, size, k, "dx")
    dy, (dw, size) = combine_backward_ref(dout, y, pos, w)
    got_dy, got_dw = moe.moe_combine_backward(dout, y, pos, pair_ids, w)
    check(got_dy, dy, name="dy")
    check(got_dw, dw, size, H, "dweights")
    one, _ = moe.moe_combine_backward(dout, y, pos, pair_ids)
    check(one, combine_backward_ref(dout, y, pos, torch.ones(T, k))[0], name="dy without weights")


def test_gradients_against_differences():
    """<dout, combine(y + v) - combine(y)> = <dy, v>, the same for the weights and for dispatch (all linear)."""
    g = gen(5)
    T, k, E, H = 40, 4, 9, 48
    ids = make_ids(g, T, k, E, 0.1).cuda()
    x, vx = rand(g, T, H), rand(g, T, H)
    d = moe.moe_dispatch(x, ids, E)
    y, vy, w, vw, dout = rand(g, T * k, H), rand(g, T * k, H), rand(g, T, k), rand(g, T, k), rand(g, T, H)
    dy, dw = moe.moe_combine_backward(dout, y, d.pos, d.pair_ids, w)
    dot = lambda a, b: (a.double() * b.double()).sum().item()  # noqa: E731
    mass = lambda a, b: (a.double() * b.double()).abs().sum().item()  # noqa: E731
    base = moe.moe_combine(y, d.pos, w)
    moved = moe.moe_combine(y + vy, d.pos, w)
    tol = 64 * 2.0 ** -24
    assert abs(dot(dout, moved) - dot(dout, base) - dot(dy, vy)) <= tol * (mass(dout, moved) + mass(dout, base)
                                                                          + mass(dy, vy)) * k
    moved = moe.moe_combine(y, d.pos, w + vw)
    assert abs(dot(dout, moved) - dot(dout, base) - dot(dw, vw)) <= tol * (mass(dout, moved) + mass(dout, base)
                                                                          + mass(dw, vw)) * k
    drows = rand(g, T * k, H)
    dx = moe.moe_dispatch_backward(drows, d.pos)
    rows = moe.moe_dispatch(vx, ids, E).rows
    assert abs(dot(drows, rows) - dot(dx, vx)) <= tol * (mass(drows, rows) + mass(dx, vx))


def test_infinities_and_nan_stay_in_their_rows():
    ids = torch.tensor([[0, 1], [1, -1], [2, 0]], dtype=torch.int32, device="cuda")
    x = torch.ones(3, 8, device="cuda", dtype=torch.bfloat16)
    x[1, 2], x[2, 3] = float("inf"), float("nan")
    d = moe.moe_dispatch(x, ids, 3)
    rows = d.rows.float().cpu()
    assert torch.isinf(rows[d.pos[1, 0].item(), 2]) and torch.isnan(rows[d.pos[2, 0].item(), 3])
    assert torch.isfinite(rows).sum().item() == 48 - 3
    y = torch.ones(6, 8, device="cuda")
    y[d.pos[0, 0].item(), 0] = float("inf")
    y[5] = float("nan")                       # the row of no pair
    one = torch.ones(3, 2, device="cuda")
    out = moe.moe_combine(y, d.pos, one)
    assert torch.isinf(out[0, 0]) and torch.isfinite(out[1:]).all() and torch.isfinite(out[0, 1:]).all()
    dy, dw = moe.moe_combine_backward(torch.ones(3, 8, device="cuda"), y, d.pos, d.pair_ids, one)
    assert torch.isfinite(dy).all() and torch.equal(dy[5], torch.zeros(8, device="cuda"))
    assert torch.isinf(dw[0, 0]) and dw[1, 1].item() == 0


def test_many_rows_of_no_pair_are_not_read():
    """The same in the kernel that many tokens take."""
    g = gen(41)
    T, k, H = 4000, 4, 512
    ids = make_ids(g, T, k, 8, 0.3).cuda()
    x, w = rand(g, T, H, dtype=torch.bfloat16), rand(g, T, k)
    d = moe.moe_dispatch(x, ids, 8)
    n = d.expert_offsets[8].item()
    y = d.rows.clone()
    y[n:] = float("nan")
    out, size = combine_ref(d.rows, d.pos, w)
    check(moe.moe_combine(y, d.pos, w), out, size, k + 1, "out")
    pos = d.pos.clone()
    pos[7, 2], pos[3999, 0] = T * k, 2 ** 31 - 1
    status_clear()
    got = moe.moe_combine(y, pos, w)
    assert status() == 2
    pos[7, 2], pos[3999, 0] = -1, -1
    assert torch.equal(got, moe.moe_combine(y, pos, w)) and status() == 0


def test_rows_past_the_matrix_are_reported():
    y = torch.ones(4, 8, device="cuda")
    pos = torch.tensor([[0, 4], [3, -1]], dtype=torch.int32, device="cuda")
    status_clear()
    out = moe.moe_combine(y, pos, torch.ones(2, 2, device="cuda"))
    assert status() == 2 and torch.equal(out, torch.ones(2, 8, device="cuda"))
    pair_ids = torch.tensor([0, -1, -1, 2], dtype=torch.int32, device="cuda")
    dy, dw = moe.moe_combine_backward(torch.ones(2, 8, device="cuda"), y, pos, pair_ids, torch.ones(2, 2, device="cuda"))
    assert status() == 2 and dw.tolist() == [[8.0, 0.0], [8.0, 0.0]]
    assert torch.equal(dy.sum(1).cpu(), torch.tensor([8.0, 0, 0, 8.0]))


def test_other_stream_and_graph():
    g = gen(21)
    T, k, E, H = 200, 4, 16, 264
    ids, x = make_ids(g, T, k, E, 0.05).cuda(), rand(g, T, H, dtype=torch.bfloat16)
    w, dout = rand(g, T, k), rand(g, T, H, dtype=torch.bfloat16)

    def step():
        d = moe.moe_dispatch(x, ids, E)
        out = moe.moe_combine(d.rows, d.pos, w)
        dy, dw = moe.moe_combine_backward(dout, d.rows, d.pos, d.pair_ids, w)
        return d.rows, out, dy, dw, moe.moe_dispatch_backward(dy, d.pos)
    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    ids.copy_(make_ids(g, T, k, E, 0.05, skew=True))
    x.copy_(rand(g, T, H, dtype=torch.bfloat16))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_rows_past_two_to_the_31_elements():
    """Row offsets that pass 32 bits: 264,000 rows of 8,200 columns."""
    T, k, H = 33000, 8, 8200
    ids = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k) % 8
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(T, device="cuda") % 251).float()[:, None].expand(T, H))
    d = moe.moe_dispatch(x, ids, 8)
    at = torch.tensor([0, 1, T * k // 2, T * k - 2, T * k - 1], device="cuda")
    want = (d.pair_ids[at].long() // k % 251).to(torch.bfloat16)
    assert torch.equal(d.rows[at], want[:, None].expand(5, H))
    dx = moe.moe_dispatch_backward(d.rows, d.pos)
    t = torch.tensor([0, T // 2, T - 1], device="cuda")
    assert torch.equal(dx[t], (x[t].float() * k).to(torch.bfloat16))
    del dx
    dy, dw = moe.moe_combine_backward(x, d.rows, d.pos, d.pair_ids)
    assert torch.equal(dy[at], want[:, None].expand(5, H))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("T,H", [(60, 1), (60, 7), (60, 17), (40, 249), (30, 250), (24, 2375), (18, 4097)])
def test_rows_between_sixteen_byte_boundaries(T, H, dtype):
    """Neighbours of a row share 16 bytes with it: what they hold (NaN here, or the gap between rows) stays theirs."""
    g = gen(T * H)
    k, E = 3, 5
    ids = make_ids(g, T, k, E, 0.1).cuda()
    x, y, dout, w = rand(g, T, H, dtype=dtype), rand(g, T * k, H, dtype=dtype), rand(g, T, H, dtype=dtype), rand(g, T, k)
    x[T // 2] = dout[T // 2] = float("nan")
    for lay in (lambda t: t, lambda t: offset_copy(t, 3), lambda t: strided_copy(t, 3, 1)):
        d = moe.moe_dispatch(lay(x), ids, E)
        offsets, pair_ids, pos = sort_ref(ids.cpu(), E)
        live = pair_ids[:int(offsets[-1])] // k
        assert torch.equal(d.rows[:len(live)].cpu().isnan(), x.cpu()[live].isnan())
        assert torch.equal(d.rows[:len(live)].cpu().nan_to_num(7.0), x.cpu()[live].nan_to_num(7.0))
        assert not d.rows[len(live):].any()
        bad = y.clone()
        r = int(torch.nonzero(pos[T // 2] >= 0)[0])
        bad[pos[T // 2, r]] = float("nan")
        out, size = combine_ref(bad, d.pos, w)
        check(moe.moe_combine(lay(bad), d.pos, w), out, size, k + 1, "out")
        dy, dw = moe.moe_combine_backward(lay(dout), lay(bad), d.pos, d.pair_ids, w)
        want, (ww, size) = combine_backward_ref(dout, bad, d.pos, w)
        check(dy, want, name="dy")
        check(dw, ww, size, H, "dweights")


def test_the_current_stream_is_torchs():
    from block_fp8_mixture_topk_gb300 import ops
    x = torch.zeros(1, device="cuda")
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert ops._stream("x", x) == torch.cuda.current_stream().cuda_stream == s.cuda_stream
