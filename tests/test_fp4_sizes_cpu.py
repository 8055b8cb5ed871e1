"""Sizes of 4-bit weights' scales: 0 for all that the packing and the products refuse, and refused where it is 0."""
import ctypes
import random

from block_fp8_mixture_topk_gb300 import ops

P = ctypes.c_void_p(0x10000)      # never read: every call below is refused
SHAPE = -2


def test_weight_scale_bytes_of_refused_sizes():
    L = ops.lib()
    good = dict(fmt=1, E=2, N=64, K=64)
    assert L.moe_fp4_weight_scale_bytes(*good.values()) == 2 * 1 * 1 * 2048
    for change in (dict(K=32800), dict(K=48), dict(E=1025), dict(N=1 << 24), dict(N=100), dict(N=1)):
        s = {**good, **change}
        assert L.moe_fp4_weight_scale_bytes(*s.values()) == 0 == ops._fp4_weight_scale_bytes(*s.values()), change
        assert L.moe_fp4_pack_scales(P, s["fmt"], s["E"], s["N"], s["K"], 0, P, None) == SHAPE, change
        assert L.moe_fp4_expert_gemm(P, P, P, s["fmt"], P, P, P, P, 10, s["E"], s["N"], s["K"], 0, 0, P, None, None) == SHAPE, change
    for change in (dict(fmt=2), dict(E=0), dict(N=0), dict(K=0), dict(E=-1), dict(N=-8), dict(K=-32)):
        assert L.moe_fp4_weight_scale_bytes(*{**good, **change}.values()) == 0, change
    assert L.moe_fp4_weight_scale_bytes(1, 1024, (1 << 24) - 8, 32768) == 0   # tiles past 2^31


def test_weight_scale_bytes_of_taken_sizes():
    L, r = ops.lib(), random.Random(2)
    for _ in range(300):
        f, E, N, K = r.randint(0, 1), r.randint(1, 64), 8 * r.randint(1, 4000), 32 * r.randint(1, 1024)
        size = E * -(-N // 128) * -(-K // 256) * (2 << f) * 512
        assert L.moe_fp4_weight_scale_bytes(f, E, N, K) == size == ops._fp4_weight_scale_bytes(f, E, N, K)
