"""4-bit rows and weights and the experts' products on them against 64-bit values."""
import pytest
import torch

import block_fp8_mixture_topk_gb300 as moe
from train_testutil import DTYPES, check, gen, half_step, ids_of, offset_copy, rand, status, status_clear, strided_copy

pytestmark = pytest.mark.gpu
FORMATS = ["mxfp4", "nvfp4"]
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def power(e):
    """2^e of whole numbers, exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def nearest(a, table):
    """Indices of the nearest entries of an ascending table, ties to the even index."""
    border = (table[1:] + table[:-1]) / 2
    low = torch.searchsorted(border, a.contiguous())                  # borders below a
    high = torch.searchsorted(border, a.contiguous(), right=True)     # borders up to a
    return torch.where(low == high, low, low + low % 2)               # on a border: the even one of the two


def quantise64(x, fmt):
    """Numbers that the 4-bit rows of x stand for, fp64 on the CPU (NaN where an infinity or NaN spreads)."""
    v = x.detach().double().cpu().reshape(x.shape[0], -1, 32 if fmt == "mxfp4" else 16)
    bad = ~torch.isfinite(v)
    if fmt == "nvfp4":
        bad = bad.any(2, keepdim=True).any(1, keepdim=True).expand_as(v)
    else:
        bad = bad.any(2, keepdim=True).expand_as(v)
    v = torch.where(bad, 0.0, v)
    top = v.abs().amax(2, keepdim=True)
    if fmt == "mxfp4":
        powers = power(torch.arange(-127, 128))
        d = powers[torch.searchsorted(powers, top / 6).clamp(max=254)]
    else:
        r = (top.amax(1, keepdim=True) / 2688).float().double()
        ratio = torch.where(r > 0, top / (6 * torch.where(r > 0, r, 1.0)), 0.0)
        d = E4M3[nearest(ratio, E4M3)] * r
    q = torch.where(d > 0, E2M1[nearest(v.abs() / torch.where(d > 0, d, 1.0), E2M1)], 0.0)
    return torch.where(bad, float("nan"), q * d * v.sign()).reshape(x.shape)


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def same(got, ref, name):
    """Equal to the last bit (of the sign of zero apart), NaN in the same places."""
    got, ref = got.cpu(), ref.to(got.dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN in other places"
    wrong = (got != ref) & ~torch.isnan(ref)
    assert not wrong.any(), f"{name}: {int(wrong.sum())} of {wrong.numel()}, first at {wrong.nonzero()[0].tolist()}"


def spread(g, rows, K, dtype, device="cuda"):
    """Rows whose magnitudes differ from column to column and row to row."""
    x = torch.randn(rows, K, generator=g) * torch.exp(torch.randn(K, generator=g)) * torch.exp(torch.randn(rows, 1, generator=g))
    return x.to(dtype).to(device)


# ---------------------------------------------------------------------------------- quantisation
SHAPES = [(1, 32), (3, 64), (8, 96), (5, 256), (7, 288), (224, 512), (225, 544), (449, 2048), (2, 7168), (31, 8192 + 32),
          (2, 32768)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_values(shape, fmt, dtype):
    x = spread(gen(1), *shape, dtype)
    rows = moe.moe_fp4_quant(x, fmt)
    same(moe.moe_fp4_dequant(rows, torch.float32), quantise64(x, fmt), "values")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
def test_result_types(dtype, fmt):
    x = spread(gen(2), 40, 352, torch.float32).clamp(-1e4, 1e4)
    ref = quantise64(x, fmt).float()
    got = moe.moe_fp4_dequant(moe.moe_fp4_quant(x, fmt), dtype)
    assert torch.equal(got.cpu(), ref.to(dtype))   # of the fp32 number


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
def test_strides_and_addresses(dtype, fmt):
    x = spread(gen(3), 37, 320, dtype)
    want = moe.moe_fp4_dequant(moe.moe_fp4_quant(x, fmt), torch.float32)
    for y in (offset_copy(x), strided_copy(x, 1), strided_copy(x, 8, 8), strided_copy(x, 5, 3)):
        got = moe.moe_fp4_quant(y, fmt)
        assert torch.equal(moe.moe_fp4_dequant(got, torch.float32), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_borders(fmt):
    """Numbers on and next to the borders between codes and between scales."""
    g = gen(4)
    base = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = []
    for scale in (1.0, 0.3331, 7.77, 2.0 ** -20, 1.0 / 3, 448 * 1.1):
        v = base[torch.randint(0, 7, (64, 64), generator=g)] * scale
        v = v * (1 + torch.randint(-2, 3, v.shape, generator=g) * 2.0 ** -23)
        v[:, ::16] = 6.0 * scale        # the block's largest
        v[::2] *= -1
        rows.append(v)
    # blocks whose largest is at a border of the e4m3 scale of a row of 2688
    for m in range(8, 16):
        v = torch.full((4, 64), 1e-3)
        v[:, 0] = 2688.0
        for i in range(1, 4):
            v[:, 16 * i] = 6 * (m + 0.5) * 2.0 ** (i - 2) * (1 + torch.arange(-2, 2) * 2.0 ** -23)
        rows.append(v)
    x = torch.cat(rows).cuda()
    same(moe.moe_fp4_dequant(moe.moe_fp4_quant(x, fmt), torch.float32), quantise64(x, fmt), "values")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("fmt", FORMATS)
def test_extremes(fmt, dtype):
    """Zero rows and groups, the smallest and largest numbers, infinities and NaN."""
    t = torch.finfo(dtype)
    x = spread(gen(5), 12, 128, torch.float32)
    x[0] = 0
    x[1, 32:64] = 0
    x[2] = t.max
    x[3] = t.smallest_normal
    x[4] = t.smallest_normal * t.eps * torch.arange(1, 129)
    x[5, :64], x[5, 64:] = t.max, t.smallest_normal
    x[6, 40] = float("inf")
    x[7, 3] = float("-inf")
    x[8, 100] = float("nan")
    x[9] = float("nan")
    x[10] = -0.0
    x[11, 1:] = 0
    x = x.clamp(-t.max, t.max).to(dtype) if dtype != torch.float32 else x
    x[6, 40], x[7, 3] = float("inf"), float("-inf")
    x = x.cuda()
    same(moe.moe_fp4_dequant(moe.moe_fp4_quant(x, fmt), torch.float32), quantise64(x, fmt), "values")


COUNTS = [[1], [0, 3, 0, 0, 1], [224, 223, 225, 0, 1], [448, 449, 5], [0, 0, 0], [2] * 300, [1, 0] * 512, [1000, 0, 700]]


@pytest.mark.parametrize("left", [0, 9])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_sorted_rows(counts, fmt, left):
    """Rows of experts keep their numbers in the experts' tiles, the rows of no expert too."""
    off = offsets_of(counts)
    x = spread(gen(6), sum(counts) + left, 96, torch.bfloat16)
    rows = moe.moe_fp4_quant(x, fmt, off)
    if x.shape[0] == 0:
        return
    same(moe.moe_fp4_dequant(rows, torch.float32), quantise64(x, fmt), "values")
    plain = moe.moe_fp4_quant(x, fmt)
    assert torch.equal(rows.codes, plain.codes)


def test_rows_keep_their_neighbours():
    """Nothing is written past the codes, the scales and the row scales."""
    for fmt in FORMATS:
        x = spread(gen(7), 230, 288, torch.bfloat16)
        L, f = moe.ops.lib(), moe.ops.FP4_FORMAT[fmt]
        size = L.moe_fp4_row_scale_bytes(f, 230, 0, 288)
        codes = torch.full((231, 144), 0xAA, dtype=torch.uint8, device="cuda")
        scales = torch.full((size + 512,), 0xAA, dtype=torch.uint8, device="cuda")
        rs = torch.full((231,), 7.0, device="cuda")
        rc = L.moe_fp4_quant(x.data_ptr(), 288, 0, f, None, 0, 230, 288, codes.data_ptr(), scales.data_ptr(),
                             rs.data_ptr() if f else None, None)
        torch.cuda.synchronize()
        assert rc == 0
        assert (codes[230] == 0xAA).all() and (scales[size:] == 0xAA).all() and rs[230] == 7.0
        want = moe.moe_fp4_quant(x, fmt)
        assert torch.equal(codes[:230], want.codes)


def test_mxfp4_weights():
    for dtype in DTYPES:
        w = spread(gen(8), 6 * 40, 160, dtype).reshape(6, 40, 160)
        q, s = moe.moe_mxfp4_quant_weight(w)
        same(weights64(q, s, None, "mxfp4").reshape(240, 160), quantise64(w.reshape(240, 160), "mxfp4"), "weights")


# -------------------------------------------------------------------------------------- products
def weights64(q, s, glob, fmt):
    """Numbers that 4-bit weights [E, N, K/2] stand for, fp64 on their device."""
    table = torch.cat([E2M1, -E2M1]).to(q.device)
    v = table[torch.stack([q & 15, q >> 4], 3).reshape(*q.shape[:2], -1).long()]
    if fmt == "mxfp4":
        scale = power(s.int() - 127)
    else:
        scale = s.view(torch.float8_e4m3fn).double() * glob.double()[:, None, None]
    return (v.reshape(*scale.shape, -1) * scale[..., None]).reshape(v.shape)


def make_weights(g, E, N, K, fmt, gate_up=False):
    """(codes, packed scales, global or None, numbers in 64 bits)."""
    w = torch.randn(E, N, K, generator=g) * torch.exp(0.5 * torch.randn(E, N, 1, generator=g))
    w = w.to(torch.bfloat16).cuda()
    if fmt == "mxfp4":
        (q, s), glob = moe.moe_mxfp4_quant_weight(w), None
    else:
        q, s, glob = moe.moe_nvfp4_quant_weight(w)
    return q, moe.moe_fp4_pack_scales(s, fmt, gate_up), glob, weights64(q, s, glob, fmt)


def steps(n):
    """fp32 half-steps of a tensor-core sum of n products: 16 of them at a time (fewer joins in these products, which
    take 64), each join truncated (two half steps) and aligned inside the step (as much again), and the scales' two."""
    return 4 * ((n + 15) // 16) + 12


def product64(a, w, ends):
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
    ([1], 0, 32, 32),
    ([0, 3, 0, 0, 1], 2, 96, 64),
    ([128, 127, 129, 0, 1], 0, 256, 256),
    ([5, 224, 64, 63, 65, 0], 3, 288, 224),
    ([225, 31, 33], 1, 160, 288),
    ([17] * 9, 0, 544, 160),
    ([700, 2], 5, 96, 1024),
    ([0, 0, 0], 7, 32, 64),
    ([2] * 300, 0, 64, 64),
    ([1, 0] * 512, 1, 32, 32),
    ([513, 1500, 0, 40, 1025], 9, 352, 544),
    ([448, 449, 2000, 97], 0, 800, 2080),
    # many items: two row tiles to one
    ([5000, 0, 449, 20000, 300, 224, 1], 5, 4096, 64),
    ([5000, 0, 449, 20000, 300, 448, 1], 5, 4096, 512),
    ([5000, 0, 449, 20000, 300, 224, 1], 0, 4096, 544),
    ([17, 25000, 0, 673, 240], 3, 4128, 1312),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[2]}-{c[3]}")
def test_product(case, fmt):
    counts, left, N, K = case
    g = gen(11)
    off = offsets_of(counts)
    ends = off.tolist()
    x = spread(g, sum(counts) + left, K, torch.bfloat16)
    q, tiles, glob, w = make_weights(g, len(counts), N, K, fmt)
    status_clear()
    rows = moe.moe_fp4_quant(x, fmt, off)
    a = moe.moe_fp4_dequant(rows, torch.float32).double()
    c, size = product64(a, w, ends)
    for dtype in DTYPES:
        if dtype == torch.float16:   # inside its range
            rows2 = moe.moe_fp4_quant(x * 1e-3, fmt, off)
            c2, size2 = product64(moe.moe_fp4_dequant(rows2, torch.float32).double(), w, ends)
            check(moe.moe_fp4_expert_gemm(rows2, q, tiles, glob, dtype), c2, size2, steps(K), "c")
        else:
            check(moe.moe_fp4_expert_gemm(rows, q, tiles, glob, dtype), c, size, steps(K), "c")
    assert status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[2]}-{c[3]}")
def test_silu_product(case, fmt):
    counts, left, N, K = case
    g = gen(12)
    off = offsets_of(counts)
    x = (torch.randn(sum(counts) + left, K, generator=g) * K ** -0.5).bfloat16().cuda()
    q, tiles, glob, w = make_weights(g, len(counts), N, K, fmt, gate_up=True)
    status_clear()
    rows = moe.moe_fp4_quant(x, fmt, off)
    c, size = product64(moe.moe_fp4_dequant(rows, torch.float32).double(), w, off.tolist())
    h, hs = silu64(c, size)
    for dtype in (torch.bfloat16, torch.float16):
        got = moe.moe_fp4_expert_gemm_silu_mul(rows, q, tiles, glob, dtype)
        check(got, h, hs, steps(K) + 8, "h")
        if dtype == torch.bfloat16 and N % 64 == 0 and x.shape[0]:
            want = moe.moe_fp4_quant(got, fmt, off)
            have = moe.moe_fp4_expert_gemm_silu_mul_quant(rows, q, tiles, glob)
            assert have.format == fmt and have.expert_offsets is off
            live = off[-1].item()
            assert torch.equal(have.codes[:live], want.codes[:live])
            values = moe.moe_fp4_dequant(have, torch.float32), moe.moe_fp4_dequant(want, torch.float32)
            assert torch.equal(values[0][:live], values[1][:live])
    assert status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_weight_for_all_rows(fmt):
    g = gen(13)
    for n in (1, 100, 1000):
        x = spread(g, n, 192, torch.float16)
        q, tiles, glob, w = make_weights(g, 1, 136, 192, fmt)
        rows = moe.moe_fp4_quant(x, fmt)
        c, size = product64(moe.moe_fp4_dequant(rows, torch.float32).double(), w, [0, n])
        check(moe.moe_fp4_expert_gemm(rows, q, tiles, glob, torch.float32), c, size, steps(192), "c")


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_row_of_nan_stays_alone(fmt):
    g = gen(14)
    off = offsets_of([30, 40])
    x = spread(g, 70, 256, torch.bfloat16)
    q, tiles, glob, _ = make_weights(g, 2, 64, 256, fmt)
    want = moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x, fmt, off), q, tiles, glob)
    x[29, 7] = float("nan")
    x[50, 200] = float("inf")
    got = moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x, fmt, off), q, tiles, glob)
    fine = torch.ones(70, dtype=torch.bool)
    fine[29] = fine[50] = False
    assert torch.isnan(got[~fine]).all() and torch.equal(got[fine], want[fine])


def test_captured_and_on_another_stream():
    g = gen(15)
    off = offsets_of([30, 0, 41])
    q, tiles, glob, _ = make_weights(g, 3, 128, 64, "nvfp4", gate_up=True)
    q2, tiles2, glob2, _ = make_weights(g, 3, 64, 64, "nvfp4")
    x = spread(g, 71, 64, torch.bfloat16)

    def step():
        h = moe.moe_fp4_expert_gemm_silu_mul_quant(moe.moe_fp4_quant(x, "nvfp4", off), q, tiles, glob)
        return moe.moe_fp4_expert_gemm(h, q2, tiles2, glob2)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(step(), want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.current_stream().wait_stream(side)
    y = spread(gen(16), 71, 64, torch.bfloat16)
    x.copy_(y)
    graph.replay()
    assert torch.equal(out, step())


@pytest.mark.parametrize("counts, N", [([300, 5, 700], 512), ([9000, 5, 18000], 4096)])
def test_results_repeat(counts, N):
    g = gen(17)
    off = offsets_of(counts)
    for fmt in FORMATS:
        q, tiles, glob, _ = make_weights(g, 3, N, 1024, fmt)
        rows = moe.moe_fp4_quant(spread(g, sum(counts), 1024, torch.bfloat16), fmt, off)
        want = moe.moe_fp4_expert_gemm(rows, q, tiles, glob)
        for _ in range(20):
            assert torch.equal(moe.moe_fp4_expert_gemm(rows, q, tiles, glob), want)


def test_offsets_out_of_order_are_reported():
    g = gen(18)
    for fmt in FORMATS:
        q, tiles, glob, _ = make_weights(g, 3, 64, 64, fmt)
        x = spread(g, 50, 64, torch.bfloat16)
        bad = torch.tensor([3, 20, 10, 60], dtype=torch.int32, device="cuda")
        good = torch.tensor([0, 20, 20, 50], dtype=torch.int32, device="cuda")
        status_clear()
        got = moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x, fmt, bad), q, tiles, glob)
        assert status() == 0x4
        assert torch.equal(got, moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x, fmt, good), q, tiles, glob))


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_launches_and_large_results(fmt):
    """More items than a cluster's table holds, results past 2^31 elements: columns and the last rows as in small calls."""
    g = gen(20)
    n, N, K = 66000, 32768, 64
    x = spread(g, n, K, torch.bfloat16)
    q, tiles, glob, _ = make_weights(g, 1, N, K, fmt)
    out = moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x, fmt), q, tiles, glob)
    assert out.numel() > 2 ** 31
    cut = q[:, :4096].contiguous(), tiles[:, :32].contiguous()
    assert torch.equal(out[:, :4096], moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x, fmt), *cut, glob))
    tail = moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x[-300:].clone(), fmt), q, tiles, glob)
    assert torch.equal(out[-300:], tail)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_past_2_31_elements(fmt):
    n, K = 70000, 32768
    x = torch.empty(n, K, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    off = torch.tensor([0, 100, 69000, n], dtype=torch.int32, device="cuda")
    rows = moe.moe_fp4_quant(x, fmt, off)
    tail = moe.moe_fp4_quant(x[-300:].clone(), fmt)
    assert torch.equal(rows.codes[-300:], tail.codes)
    assert torch.equal(moe.moe_fp4_dequant(rows)[-300:], moe.moe_fp4_dequant(tail))


def test_borders_of_16_bit_rows():
    """Every largest magnitude of a bf16 row with every number below it, and many of fp16's: quotients that nvfp4's borders meet."""
    for dtype, bits in ((torch.bfloat16, 7), (torch.float16, 10)):
        for start in range(0, 2 ** bits, 1 if bits == 7 else 13):
            top = 1 + start / 2 ** bits
            below = (1 + torch.arange(2 ** bits, dtype=torch.float64) / 2 ** bits)[None] * 2.0 ** -torch.arange(0, 8)[:, None]
            v = below.reshape(-1)
            v = v[v <= top]
            v = torch.cat([v, torch.zeros(-len(v) % 64)])[:32768]
            x = torch.stack([v, v.flip(0)])
            x = torch.cat([x, torch.zeros(2, 64)], 1)[:, :32768 - 64] if x.shape[1] > 32768 - 64 else torch.cat([x, torch.zeros(2, 64)], 1)
            x[:, -1] = top
            x = x.to(dtype).cuda()
            same(moe.moe_fp4_dequant(moe.moe_fp4_quant(x, "nvfp4"), torch.float32), quantise64(x, "nvfp4"), f"{dtype} {top}")


def test_half_step_of_a_product_of_ones():
    """Products of numbers that 4 bits hold exactly are exact."""
    x = torch.ones(40, 512, dtype=torch.bfloat16, device="cuda")
    for fmt in FORMATS:
        q, tiles, glob, w = make_weights(gen(19), 1, 40, 512, fmt)
        got = moe.moe_fp4_expert_gemm(moe.moe_fp4_quant(x, fmt), q, tiles, glob, torch.float32)
        check(got, (moe.moe_fp4_dequant(moe.moe_fp4_quant(x, fmt), torch.float32).double() @ w[0].T), w[0].abs().sum(1)[None].expand(40, 40),
              steps(512), "ones")
    assert half_step(torch.float32) == 2.0 ** -24


def test_rows_are_checked_at_each_call():
    """Rows of which a tensor was given other memory are refused, those that these functions made as well."""
    rows = moe.moe_fp4_quant(torch.ones(300, 512, dtype=torch.bfloat16, device="cuda"), "nvfp4")
    moe.moe_fp4_dequant(rows)
    for name, other in (("codes", rows.codes[:200].clone()), ("scales", rows.scales[:512].clone()),
                        ("row_scale", rows.row_scale[:10].clone())):
        part = getattr(rows, name)
        kept = part.data
        part.data = other
        with pytest.raises(ValueError):
            moe.moe_fp4_dequant(rows)
        part.data = kept
    moe.moe_fp4_dequant(rows)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids_of)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [2080, 8192, 8224, 9216, 16416, 20000, 32736])
def test_long_rows(K, fmt, dtype):
    """Rows of every share of a block's threads."""
    x = spread(gen(22), 5, K, dtype)
    rows = moe.moe_fp4_quant(x.cuda(), fmt)
    assert torch.equal(moe.moe_fp4_dequant(rows, torch.float32).cpu(), quantise64(x, fmt).float())
