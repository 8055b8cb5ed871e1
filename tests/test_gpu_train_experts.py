"""The experts' 16-bit products and their gradients against 64-bit values."""
import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from train_testutil import check, gen, ids_of, rand, status, status_clear, strided_copy

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def steps(n):
    """fp32 half-steps of a tensor-core sum of n products: 16 of them at a time, each join truncated (two half
    steps) and aligned inside the step (as much again)."""
    return 4 * ((n + 15) // 16) + 8


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def product64(a, w, ends):
    """(a @ w[e]^T, the same of magnitudes) per expert in 64 bits; zero past the last expert."""
    a, w = a.double(), w.double()
    out = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64, device=a.device)
    size = torch.zeros_like(out)
    for e in range(w.shape[0]):
        lo, hi = ends[e], ends[e + 1]
        out[lo:hi] = a[lo:hi] @ w[e].T
        size[lo:hi] = a[lo:hi].abs() @ w[e].abs().T
    return out, size


def silu64(c, size):
    gate, up = c.chunk(2, 1)
    sg, su = size.chunk(2, 1)
    h = torch.nn.functional.silu(gate) * up
    # |d silu| <= 1.1: the products' errors through the activation
    return h, 1.1 * sg * up.abs() + torch.nn.functional.silu(gate).abs() * su + 4 * h.abs()


CASES = [  # rows per expert, rows of no expert, N, K
    ([1], 0, 16, 8),
    ([0, 3, 0, 0, 1], 2, 48, 72),
    ([128, 127, 129, 0, 1], 0, 256, 64),
    ([5, 300, 64, 63, 65, 0], 3, 272, 200),
    ([17] * 9, 0, 528, 136),
    ([700, 2], 5, 96, 1024),
    ([0, 0, 0], 7, 32, 64),
    ([2] * 300, 0, 64, 64),
    ([1, 0] * 512, 1, 16, 16),
    ([513, 1500, 0, 40, 1025], 9, 336, 328),      # several tiles of rows
    ([1030], 0, 1040, 72),
    ([257, 2000, 700], 0, 272, 16),
]


def inputs(case, dtype, seed):
    counts, left, N, K = case
    g = gen(seed)
    rows = sum(counts) + left
    off = offsets_of(counts)
    return (off, off.tolist(), rand(g, rows, K, dtype=dtype), rand(g, len(counts), N, K, dtype=dtype, std=0.1),
            rand(g, rows, N, dtype=dtype, std=0.5), rand(g, rows, 2 * K, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[2]}-{c[3]}")
def test_product(case, dtype):
    off, ends, a, w, _, _ = inputs(case, dtype, 1)
    status_clear()
    c, size = product64(a, w, ends)
    check(moe.moe_expert_gemm(a, w, off), c, size, steps(case[3]), "c")
    h, gu = moe.moe_expert_gemm_silu_mul(a, w, off)
    check(gu, c, size, steps(case[3]), "gate_up")
    h64, hs = silu64(c, size)
    check(h, h64, hs, steps(case[3]) + 8, "h")
    h2, none = moe.moe_expert_gemm_silu_mul(a, w, off, save_gate_up=False)
    assert none is None and torch.equal(h, h2)
    assert status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[2]}-{c[3]}")
def test_rows_gradient(case, dtype):
    off, ends, _, w, dc, gu = inputs(case, dtype, 2)
    da, size = product64(dc, w.transpose(1, 2), ends)
    check(moe.moe_expert_gemm_dgrad(dc, w, off), da, size, steps(case[2]), "da")
    gate, up = gu.double().chunk(2, 1)
    s = torch.sigmoid(gate)
    kg, ku = up * s * (1 + gate * (1 - s)), gate * s
    # the factor 1 + gate * (1 - s) may cancel: its parts count
    mg = up.abs() * s * (1 + gate.abs() * (1 - s))
    ref = torch.cat([da * kg, da * ku], 1)
    err = steps(case[2]) * torch.cat([size * kg.abs(), size * ku.abs()], 1) + 16 * torch.cat([da.abs() * mg,
                                                                                            (da * ku).abs()], 1)
    check(moe.moe_expert_gemm_dgrad(dc, w, off, gate_up=gu), ref, err, 1, "dgate, dup")


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[2]}-{c[3]}")
def test_weights_gradient(case, dtype):
    off, ends, a, _, dc, _ = inputs(case, dtype, 3)
    dw = moe.moe_expert_gemm_wgrad(dc, a, off)
    ref, size = torch.zeros(dw.shape, dtype=torch.float64), torch.zeros(dw.shape, dtype=torch.float64)
    x, y = a.double().cpu(), dc.double().cpu()
    for e in range(dw.shape[0]):
        lo, hi = ends[e], ends[e + 1]
        ref[e], size[e] = y[lo:hi].T @ x[lo:hi], y[lo:hi].abs().T @ x[lo:hi].abs()
    check(dw, ref, size, steps(max(case[0])), "dw")


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
def test_large_tiles_many_items(dtype, long):
    """Every SM takes several tiles of each product (accumulators alternate, the ring wraps), K and
    N past several blocks."""
    g = torch.Generator(device="cuda").manual_seed(6)
    counts = [500, 0, 1400, 129, 300, 1, 700, 640] if not long else [3000, 0, 700, 257, 9000, 1, 2000, 640, 513]
    off, rows, N, K = offsets_of(counts), sum(counts), 1552, 1096
    ends = off.tolist()
    a = torch.randn(rows, K, generator=g, device="cuda").to(dtype)
    w = (torch.randn(len(counts), N, K, generator=g, device="cuda") * 0.1).to(dtype)
    dc = (torch.randn(rows, N, generator=g, device="cuda") * 0.5).to(dtype)
    c, size = product64(a, w, ends)
    check(moe.moe_expert_gemm(a, w, off), c, size, steps(K), "c")
    h, gu = moe.moe_expert_gemm_silu_mul(a, w, off)
    h64, hs = silu64(c, size)
    check(gu, c, size, steps(K), "gate_up")
    check(h, h64, hs, steps(K) + 8, "h")
    da, size = product64(dc, w.transpose(1, 2), ends)
    check(moe.moe_expert_gemm_dgrad(dc, w, off), da, size, steps(N), "da")
    dw = moe.moe_expert_gemm_wgrad(dc, a, off)
    for e in range(len(counts)):
        x, y = a[ends[e]:ends[e + 1]].double(), dc[ends[e]:ends[e + 1]].double()
        check(dw[e], y.T @ x, y.abs().T @ x.abs(), steps(max(counts)), f"dw {e}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
def test_neighbours_do_not_leak(dtype):
    """A NaN or an infinity in one expert's rows reaches neither another's product nor its weights' gradient, nor do
    the rows of no expert."""
    g = gen(7)
    counts, N, K = [3, 70, 30], 64, 48
    off, rows = offsets_of(counts), sum(counts) + 4
    a, w, dc = rand(g, rows, K, dtype=dtype), rand(g, 3, N, K, dtype=dtype), rand(g, rows, N, dtype=dtype)
    clean = (moe.moe_expert_gemm(a, w, off), moe.moe_expert_gemm_dgrad(dc, w, off), moe.moe_expert_gemm_wgrad(dc, a, off))
    a[10, 5], a[103], dc[20, 7], dc[104] = float("nan"), float("inf"), float("-inf"), float("nan")
    c, da, dw = moe.moe_expert_gemm(a, w, off), moe.moe_expert_gemm_dgrad(dc, w, off), moe.moe_expert_gemm_wgrad(dc, a, off)
    keep = torch.ones(rows, dtype=torch.bool)
    keep[10] = False
    assert torch.equal(c[keep], clean[0][keep]) and torch.isnan(c[10]).all()
    keep[10], keep[20] = True, False
    assert torch.equal(da[keep], clean[1][keep]) and not torch.isfinite(da[20]).any()
    assert torch.equal(dw[[0, 2]], clean[2][[0, 2]]) and torch.isnan(dw[1]).any()
    assert c[103:].abs().sum().item() == 0 and da[103:].abs().sum().item() == 0


def test_strided_rows():
    g = gen(9)
    off = offsets_of([40, 7, 0, 100])
    a, w, dc = (rand(g, 147, 72, dtype=torch.bfloat16), rand(g, 4, 48, 72, dtype=torch.bfloat16),
                rand(g, 147, 48, dtype=torch.bfloat16))
    gu = rand(g, 147, 144, dtype=torch.bfloat16)
    for lay in (lambda t: strided_copy(t, 24, 8), lambda t: strided_copy(t, 8)):
        assert torch.equal(moe.moe_expert_gemm(lay(a), w, off), moe.moe_expert_gemm(a, w, off))
        assert torch.equal(moe.moe_expert_gemm_dgrad(lay(dc), w, off, gate_up=lay(gu)),
                           moe.moe_expert_gemm_dgrad(dc, w, off, gate_up=gu))
        assert torch.equal(moe.moe_expert_gemm_wgrad(lay(dc), lay(a), off), moe.moe_expert_gemm_wgrad(dc, a, off))


def test_no_rows():
    off = offsets_of([0, 0])
    a, w, dc = (torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 32, 16, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda"))
    assert moe.moe_expert_gemm(a, w, off).shape == (0, 32)
    assert moe.moe_expert_gemm_dgrad(dc, w, off).shape == (0, 16)
    assert torch.equal(moe.moe_expert_gemm_wgrad(dc, a, off), torch.zeros(2, 32, 16, dtype=torch.bfloat16, device="cuda"))


def test_offsets_out_of_range_are_clamped_and_reported():
    g = gen(12)
    a, w = rand(g, 20, 16, dtype=torch.bfloat16), rand(g, 3, 32, 16, dtype=torch.bfloat16)
    status_clear()
    bad = torch.tensor([0, 8, 400, 400], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 8, 20, 20], dtype=torch.int32, device="cuda")
    assert torch.equal(moe.moe_expert_gemm(a, w, bad), moe.moe_expert_gemm(a, w, good))
    assert status() == 4
    moe.moe_expert_gemm(a, w, torch.tensor([0, 12, 5, 20], dtype=torch.int32, device="cuda"))
    assert status() == 4
    moe.moe_expert_gemm_wgrad(rand(g, 20, 32, dtype=torch.bfloat16), a, torch.tensor([0, -4, 5, 20], dtype=torch.int32, device="cuda"))
    assert status() == 4


def test_gradients_against_differences():
    """<dc, product(v, w)> = <da, v> and <dw, v> (linear), and through SiLU(gate)*up against central
    differences of the formula in 64 bits; the kernels' results are rounded to bf16 once (at most
    2^-8 of each term)."""
    g = gen(13)
    off = offsets_of([30, 0, 65])
    ends, N, K = off.tolist(), 64, 48
    a, va, w, vw, dc = (rand(g, 95, K, dtype=torch.bfloat16), rand(g, 95, K, dtype=torch.bfloat16),
                        rand(g, 3, N, K, dtype=torch.bfloat16), rand(g, 3, N, K, dtype=torch.bfloat16),
                        rand(g, 95, N, dtype=torch.bfloat16))
    da, dw = moe.moe_expert_gemm_dgrad(dc, w, off), moe.moe_expert_gemm_wgrad(dc, a, off)
    dot = lambda x, y: (x.double() * y.double()).sum().item()  # noqa: E731
    mass = lambda x, y: (x.double() * y.double()).abs().sum().item()  # noqa: E731
    assert abs(dot(da, va) - dot(dc, product64(va, w, ends)[0])) <= 2.0 ** -8 * mass(da, va)
    assert abs(dot(dw, vw) - dot(dc, product64(a, vw, ends)[0])) <= 2.0 ** -8 * mass(dw, vw)
    gu, vgu = rand(g, 95, 2 * K, dtype=torch.bfloat16), rand(g, 95, 2 * K, dtype=torch.bfloat16)
    w2 = rand(g, 3, N, K, dtype=torch.bfloat16)

    def loss(s):
        x = gu.double() + s * vgu.double()
        h = torch.nn.functional.silu(x[:, :K]) * x[:, K:]
        return dot(dc, product64(h, w2, ends)[0])
    dgu = moe.moe_expert_gemm_dgrad(dc, w2, off, gate_up=gu)
    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs(dot(dgu, vgu) - want) <= 2.0 ** -8 * mass(dgu, vgu)


def test_other_stream_and_graph():
    g = gen(14)
    off = offsets_of([100, 30, 0, 70])
    a, w, dc = (rand(g, 200, 64, dtype=torch.bfloat16), rand(g, 4, 96, 64, dtype=torch.bfloat16),
                rand(g, 200, 96, dtype=torch.bfloat16))

    def step():
        h, gu = moe.moe_expert_gemm_silu_mul(a, w, off)
        return (h, gu, moe.moe_expert_gemm(a, w, off), moe.moe_expert_gemm_dgrad(dc, w, off),
                moe.moe_expert_gemm_wgrad(dc, a, off))
    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    off.copy_(offsets_of([0, 150, 50, 0]))
    a.copy_(rand(g, 200, 64, dtype=torch.bfloat16))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, step()))


@pytest.mark.parametrize("bad", [[0, 12, 5, 20], [5, 8, 13, 20], [3, 3, 3, 3], [-7, 4, 4, 20], [0, 400, -1, 20],
                                 [20, 10, 5, 0], [2 ** 31 - 1, -2 ** 31, 7, 19], [9, 0, 20, 20]],
                         ids=lambda b: "-".join(map(str, b)))
def test_offsets_out_of_order_are_repaired(bad):
    """Every row up to the last offset has one expert: 0 in place of the first offset, the running maximum of the
    others.  All forms equal those of the repaired offsets, in the rows of no expert too."""
    g = gen(15)
    rows, N, K = 20, 32, 16
    a, w = rand(g, rows, K, dtype=torch.bfloat16), rand(g, 3, N, K, dtype=torch.bfloat16)
    dc, gu = rand(g, rows, N, dtype=torch.bfloat16), rand(g, rows, 2 * K, dtype=torch.bfloat16)
    good = [0]
    for o in bad[1:]:
        good.append(max(good[-1], min(max(o, 0), rows)))
    bad, good = (torch.tensor(o, dtype=torch.int32, device="cuda") for o in (bad, good))

    def forms(off):
        h, c = moe.moe_expert_gemm_silu_mul(a, w, off)
        return (moe.moe_expert_gemm(a, w, off), h, c, moe.moe_expert_gemm_dgrad(dc, w, off),
                moe.moe_expert_gemm_dgrad(dc, w, off, gate_up=gu), moe.moe_expert_gemm_wgrad(dc, a, off))
    status_clear()
    want = forms(good)
    assert status() == 0
    for n in (N, N // 2, K, 2 * K):   # memory that the results take next holds NaN
        torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = forms(bad)
    assert status() == 4
    for name, x, y in zip(("c", "h", "gate_up", "da", "dgate_up", "dw"), got, want):
        assert torch.equal(x, y), name


def test_results_past_two_to_the_31_elements():
    """Offsets that pass 32 bits in rows, weights and results: the last rows and the last expert equal those of a
    call of their own."""
    g = torch.Generator(device="cuda").manual_seed(8)
    rows, N, K, last = 540000, 4096, 16, 1000
    off = torch.tensor([0, 300000, rows - last, rows], dtype=torch.int32, device="cuda")
    end = torch.tensor([0, 0, 0, last], dtype=torch.int32, device="cuda")
    a = torch.randn(rows, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(3, N, K, generator=g, device="cuda").bfloat16()
    c = moe.moe_expert_gemm(a, w, off)
    assert c.numel() > 2 ** 31 and torch.equal(c[-last:], moe.moe_expert_gemm(a[-last:], w, end))
    da = moe.moe_expert_gemm_dgrad(c, w, off)
    assert torch.equal(da[-last:], moe.moe_expert_gemm_dgrad(c[-last:], w, end))
    w2 = torch.randn(3, K, N, generator=g, device="cuda").bfloat16()
    dc = torch.randn(rows, K, generator=g, device="cuda").bfloat16()
    gu = torch.cat([c, c.flip(0)], 1)                                    # 2^32 elements
    dgu = moe.moe_expert_gemm_dgrad(dc, w2, off, gate_up=gu)
    assert torch.equal(dgu[-last:], moe.moe_expert_gemm_dgrad(dc[-last:], w2, end, gate_up=gu[-last:]))
    del c, gu, dgu
    h, gu = moe.moe_expert_gemm_silu_mul(a, w, off)
    h1, gu1 = moe.moe_expert_gemm_silu_mul(a[-last:], w, end)
    assert torch.equal(h[-last:], h1) and torch.equal(gu[-last:], gu1)
    del h, gu
    E, N, K, n = 40, 8192, 7176, 70                                      # 2.4e9 weights
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * n
    a, dc = (torch.randn(E * n, m, generator=g, device="cuda").bfloat16() for m in (K, N))
    dw = moe.moe_expert_gemm_wgrad(dc, a, off)
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for e in (0, E - 1):
        at = slice(e * n, e * n + n)
        assert torch.equal(dw[e:e + 1], moe.moe_expert_gemm_wgrad(dc[at], a[at], one))
    b = torch.randn(E * 4, K, generator=g, device="cuda").bfloat16()     # weights that are read so far out
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * 4
    c = moe.moe_expert_gemm(b, dw, off)
    one = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    assert torch.equal(c[-4:], moe.moe_expert_gemm(b[-4:], dw[-1:].contiguous(), one))
