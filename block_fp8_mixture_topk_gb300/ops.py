"""ctypes binding of libmoefp8 (argument marshalling only).

Function names and argument order follow the C ABI; tensors are torch CUDA
tensors (bf16 as torch.bfloat16, e4m3 codes as torch.uint8 or
torch.float8_e4m3fn) of the current device, launched on torch's current stream.
"""
from __future__ import annotations

import array
import ctypes
import dataclasses
import os
import threading
import warnings

import torch

from . import build as _build

MOE_BLOCK_M = 128
MOE_WEIGHTS_NK, MOE_WEIGHTS_TILED, MOE_WEIGHTS_NVFP4 = 0, 1, 2
NVFP4_UNIT_BYTES = 16 * 64 + 16 * 8   # one 16-row slab x one 128-wide K block: codes, then block scales
# fp32 amax/448; that scale rounded up to a power of two (FLOAT32_CEIL_UE8M0); the same UE8M0 scales in
# the packed scale-factor tiles of the block-scaled MMA (MOE_SCALE_UE8M0_PACKED)
# the same UE8M0 scales in the packed scale-factor tiles of the block-scaled MMA (MOE_SCALE_UE8M0_PACKED);
# MXFP8: 1x32 groups and blocks along K with UE8M0 scales, on the block-scaled MMA (MOE_SCALE_MXFP8)
SCALE_FMT = {"f32": 0, "ue8m0": 1, "ue8m0_packed": 2, "mxfp8": 3}
_PACKED_SCALES = ("ue8m0_packed", "mxfp8")
SCORING = {"softmax": 0, "sigmoid": 1}
EPILOGUE = {"store": 0, "silu_mul_quant": 1, "weighted_scatter": 2, "weighted_rows": 3, "weighted_pairs_bf16": 4}

_ERRORS = {-1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED_SHAPE", -3: "MOE_ERR_WORKSPACE_TOO_SMALL",
           -4: "MOE_ERR_CUDA", -5: "MOE_ERR_DEVICE"}


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {_ERRORS.get(code, code)}")
        self.code = code


class _RoutingParams(ctypes.Structure):
    _fields_ = [("scoring", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("routed_scaling", ctypes.c_float), ("bias", ctypes.c_void_p)]


class _Epilogue(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("topk", ctypes.c_int32), ("out_f32", ctypes.c_void_p),
                ("out_q", ctypes.c_void_p), ("out_scale", ctypes.c_void_p),
                ("out_scale_row_stride", ctypes.c_int64), ("out_scale_kb_stride", ctypes.c_int64),
                ("sorted_pair_ids", ctypes.c_void_p), ("topk_weights", ctypes.c_void_p),
                ("num_pairs", ctypes.c_int64), ("out_bf16", ctypes.c_void_p), ("b_layout", ctypes.c_int32),
                ("scale_fmt", ctypes.c_int32)]


class _ForwardOptions(ctypes.Structure):
    _fields_ = [("weight_layout", ctypes.c_int32), ("scale_fmt", ctypes.c_int32), ("decode_path", ctypes.c_int32)]


# MOE_DECODE_*: which kernels run the expert GEMMs of a small step
DECODE_PATH = {"auto": 0, "off": 1, "on": 2}


@dataclasses.dataclass
class RoutingParams:
    """Router options of the C ABI's moe_routing_params (bias: CUDA fp32 [E] or None)."""
    scoring: str = "softmax"
    n_group: int = 1
    topk_group: int = 1
    routed_scaling: float = 1.0
    bias: torch.Tensor | None = None

    def to_c(self) -> _RoutingParams:
        return _RoutingParams(SCORING[self.scoring], self.n_group, self.topk_group, float(self.routed_scaling),
                              _ptr(self.bias))


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """The loaded libmoefp8 (built on first use if absent; raises if that fails)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB_PATH):
                _build.build()
            L = ctypes.CDLL(_build.LIB_PATH)
            P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            F = ctypes.c_float
            sig = {
                "moe_route_topk": ([P, I, I, I, I, P, P, P, P], I),
                "moe_max_padded_rows": ([I, I, I, I], I64),
                "moe_max_tiles": ([I, I, I, I], I64),
                "moe_align_permute_workspace_size": ([I, I, I], SZ),
                "moe_align_permute": ([P, I, I, I, I, P, P, P, P, P, P, P, P, SZ, P], I),
                "moe_align_permute_noalloc": ([P, I, I, I, I, P, P, P, P, P, P, P, P], I),
                "fp8_group_quant": ([P, I, I, I, P, P, P], I),
                "fp8_group_quant_ex": ([P, I, I, I, P, P, I, P], I),
                "fp8_block_quant_weight_ex": ([P, I, I, I, P, P, I, P], I),
                "fp8_block_quant_weight": ([P, I, I, I, P, P, P], I),
                "fp8_block_grouped_gemm": ([P, P, I64, I64, I64, P, P, I, I, I, P, P, P, I64, P, P], I),
                "moe_fp8_block_workspace_size": ([I, I, I, I, I], SZ),
                "moe_fp8_block_forward_kernel_count": ([I, I, I, I, I], I),
                "moe_fp8_block_forward_kernel_count_ex": ([I, I, I, I, I, P, P], I),
                "moe_fp8_block_decode_path": ([I, I, I, I, I], I),
                "moe_fp8_block_pair_path": ([I, I, I, I, I], I),
                "moe_fp8_block_forward": ([P, P, P, P, P, P, I, I, I, I, I, I, P, P, SZ, P, P], I),
                "moe_fp8_block_forward_packed": ([P, P, P, P, P, P, I, I, I, I, I, I, P, P, SZ, P, P], I),
                "moe_fp8_block_forward_ex": ([P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, SZ, P, P, P], I),
                "moe_fp8_block_pack_weights": ([P, I, I, I, P, P], I),
                "moe_packed_scale_bytes": ([I64, I], SZ),
                "moe_fp8_block_pack_scales": ([P, I, I, I, P, P], I),
                "moe_mxfp8_packed_scale_bytes": ([I64, I], SZ),
                "moe_mxfp8_quant_weight": ([P, I, I, I, P, P, P], I),
                "moe_mxfp8_pack_scales": ([P, I64, I, P, P], I),
                "moe_nvfp4_quant_weight": ([P, I, I, I, P, P, P, P], I),
                "moe_nvfp4_packed_bytes": ([I, I, I], SZ),
                "moe_nvfp4_pack_weights": ([P, P, I, I, I, P, P], I),
                "moe_fp8_block_masked_workspace_size": ([I, I, I, I], SZ),
                "moe_fp8_block_forward_masked": ([P, P, P, P, P, P, I, I, I, I, P, P, SZ, P, P], I),
                "moe_unpermute_sum": ([P, I64, P, I, I, I, P, P], I),
                "moe_combine_pairs": ([P, P, I, I, I, P, P], I),
                "moe_dispatch_workspace_size": ([I, I, I], SZ),
                "moe_dispatch": ([P, I64, I, P, I, I, I, I, P, P, P, P, P, SZ, P], I),
                "moe_dispatch_backward": ([P, I64, I, P, I, I, I, I64, P, P], I),
                "moe_combine": ([P, I64, I, P, P, I, I, I, I64, P, P], I),
                "moe_combine_backward": ([P, I64, P, I64, I, P, P, P, I, I, I, I64, P, P, P], I),
                "moe_pre_norm": ([P, I64, I, P, I, F, F, I, I, P, P, P], I),
                "moe_norm_backward_workspace_size": ([I, I], SZ),
                "moe_pre_norm_backward": ([P, I64, P, I64, I, P, I, F, P, P, I64, I, I, P, P, P, SZ, P], I),
                "moe_post_norm": ([P, I64, P, I64, I, P, I, I, P, P, P, P, P], I),
                "moe_post_norm_backward": ([P, I64, P, I64, I, P, P, I, I, P, P, P, P, P, SZ, P], I),
                "moe_expert_gemm": ([P, I64, I, P, P, I64, I, I, I, I, P, P, P], I),
                "moe_expert_gemm_dgrad": ([P, I64, I, P, P, I64, I, I, I, P, I64, P, P], I),
                "moe_expert_gemm_wgrad": ([P, I64, P, I64, I, P, I64, I, I, I, P, P], I),
                "moe_clip_grads_workspace_size": ([I], SZ),
                "moe_clip_grads": ([P, P, P, P, I, I, F, F, P, P, SZ, P], I),
                "moe_get_device_status": ([P, I], I),
                "moe_selftest_bounded_wait": ([I, P], I),
                "moe_error_string": ([I], ctypes.c_char_p),
                "moe_device_supported": ([], I),
            }
            for name, (args, res) in sig.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
            _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


try:   # a third of the time of the public ones, which counts in a step of one token
    _device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
except AttributeError:
    _device = torch.cuda.current_device

    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _stream(names="", *operands):
    """The current stream of the current device, as the C ABI takes it.  An operand of another device (`names` in
    their order, None for one that is not given) is refused: the kernel would run beside the stream that
    orders it, on memory that its GPU may not reach."""
    device = _device()
    for t in operands:
        if t is not None and t.get_device() != device:
            at = [x is t for x in operands].index(True)
            raise ValueError(f"{names.split()[at]} is on {t.device}, but the current device is cuda:{device}")
    return _raw_stream(device)


def _check(name, rc):
    if rc != 0:
        raise MoeError(name, rc)


def _codes(t: torch.Tensor) -> torch.Tensor:
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"e4m3 codes must be uint8 or float8_e4m3fn, got {t.dtype}")
    return t


def _cuda(t, dtype=None, name="tensor"):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def moe_device_supported() -> bool:
    return bool(lib().moe_device_supported())


def moe_max_padded_rows(T, topk, E, block_m=MOE_BLOCK_M) -> int:
    return int(lib().moe_max_padded_rows(T, topk, E, block_m))


def moe_max_tiles(T, topk, E, block_m=MOE_BLOCK_M) -> int:
    return int(lib().moe_max_tiles(T, topk, E, block_m))


def moe_route_topk(logits, topk, renormalize=True, routing: RoutingParams | None = None):
    """Top-k routing: returns (ids int32 [T,k], weights fp32 [T,k])."""
    _cuda(logits, torch.float32, "logits")
    T, E = logits.shape
    ids = torch.empty(T, topk, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, topk, dtype=torch.float32, device=logits.device)
    rp = routing.to_c() if routing else None
    rc = lib().moe_route_topk(_ptr(logits), T, E, topk, int(bool(renormalize)),
                              ctypes.byref(rp) if rp else None, _ptr(ids), _ptr(w), _stream("logits", logits))
    _check("moe_route_topk", rc)
    return ids, w


def moe_align_permute(topk_ids, num_experts, block_m=MOE_BLOCK_M):
    """Sort pairs by expert; returns a dict of the C ABI's outputs."""
    _cuda(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    dev = topk_ids.device
    rows = moe_max_padded_rows(T, k, num_experts, block_m)
    tiles = moe_max_tiles(T, k, num_experts, block_m)
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(expert_offsets=torch.empty(num_experts + 1, **i32),
               padded_offsets=torch.empty(num_experts + 1, **i32),
               sorted_pair_ids=torch.full((max(rows, 1),), -1, **i32), pos=torch.empty(max(T * k, 1), **i32),
               tile_expert=torch.empty(max(tiles, 1), **i32), tile_row0=torch.empty(max(tiles, 1), **i32),
               num_tiles=torch.empty(1, **i32))
    wsb = int(lib().moe_align_permute_workspace_size(T, k, num_experts))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    rc = lib().moe_align_permute(_ptr(topk_ids), T, k, num_experts, block_m, _ptr(out["expert_offsets"]),
                                 _ptr(out["padded_offsets"]), _ptr(out["sorted_pair_ids"]), _ptr(out["pos"]),
                                 _ptr(out["tile_expert"]), _ptr(out["tile_row0"]), _ptr(out["num_tiles"]),
                                 _ptr(ws), wsb, _stream("topk_ids", topk_ids))
    _check("moe_align_permute", rc)
    out["max_rows"], out["max_tiles"] = rows, tiles
    return out


def moe_packed_scale_bytes(rows, K) -> int:
    """Bytes of the packed UE8M0 scale tiles of a [rows, K] operand."""
    return int(lib().moe_packed_scale_bytes(rows, K))


def fp8_group_quant(x, scale_fmt="f32"):
    """1x128 group quantisation of bf16 [rows, cols]: returns (codes uint8, scales fp32 [rows, cols/128]).
    scale_fmt: "f32" (amax/448), "ue8m0" (rounded up to a power of two), "ue8m0_packed" (the same
    scales as packed UE8M0 tiles: a uint8 tensor of moe_packed_scale_bytes(rows, cols) bytes) or
    "mxfp8" (groups of 32: the UE8M0 scale bytes, uint8 [rows, cols/32])."""
    _cuda(x, torch.bfloat16, "x")
    rows, cols = x.shape
    q = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
    if scale_fmt == "ue8m0_packed":
        s = torch.zeros(max(moe_packed_scale_bytes(rows, cols), 16), dtype=torch.uint8, device=x.device)
    elif scale_fmt == "mxfp8":
        s = torch.empty(rows, max(cols // 32, 1), dtype=torch.uint8, device=x.device)
    else:
        s = torch.empty(rows, max(cols // 128, 1), dtype=torch.float32, device=x.device)
    rc = lib().fp8_group_quant_ex(_ptr(x), rows, cols, cols, _ptr(q), _ptr(s), SCALE_FMT[scale_fmt], _stream("x", x))
    _check("fp8_group_quant", rc)
    return q, s


def fp8_block_quant_weight(w, scale_fmt="f32"):
    """128x128 block quantisation of bf16 [E, N, K]: returns (codes uint8 [E,N,K], scales [E,N/128,K/128])."""
    _cuda(w, torch.bfloat16, "w")
    E, N, K = w.shape
    q = torch.empty(E, N, K, dtype=torch.uint8, device=w.device)
    s = torch.empty(E, max(N // 128, 1), max(K // 128, 1), dtype=torch.float32, device=w.device)
    rc = lib().fp8_block_quant_weight_ex(_ptr(w), E, N, K, _ptr(q), _ptr(s), SCALE_FMT[scale_fmt], _stream("w", w))
    _check("fp8_block_quant_weight", rc)
    return q, s


def moe_fp8_block_pack_scales(s):
    """UE8M0 (power-of-two) block scales fp32 [E, N/128, K/128] -> the packed scale tiles of the
    block-scaled GEMMs, uint8 [E, N/128, ceil(K/512), 512] (load-time, once)."""
    _cuda(s, torch.float32, "s")
    E, NB, KB = s.shape
    out = torch.empty(E, NB, (KB + 3) // 4, 512, dtype=torch.uint8, device=s.device)
    _check("moe_fp8_block_pack_scales", lib().moe_fp8_block_pack_scales(_ptr(s), E, NB * 128, KB * 128, _ptr(out),
                                                                          _stream("s", s)))
    return out


def moe_mxfp8_quant_weight(w):
    """MXFP8 quantisation of bf16 expert weights [E, N, K]: returns (codes uint8 [E, N, K], UE8M0
    scale bytes uint8 [E, N, K/32]) (load-time)."""
    _cuda(w, torch.bfloat16, "w")
    E, N, K = w.shape
    q = torch.empty(E, N, K, dtype=torch.uint8, device=w.device)
    s = torch.empty(E, N, max(K // 32, 1), dtype=torch.uint8, device=w.device)
    _check("moe_mxfp8_quant_weight", lib().moe_mxfp8_quant_weight(_ptr(w), E, N, K, _ptr(q), _ptr(s), _stream("w", w)))
    return q, s


def moe_mxfp8_packed_scale_bytes(rows, K) -> int:
    return int(lib().moe_mxfp8_packed_scale_bytes(rows, K))


def moe_mxfp8_pack_scales(s):
    """UE8M0 scale bytes [..., rows, K/32] (uint8; leading dimensions folded into rows, a multiple of
    128) -> the MXFP8 packed scale tiles, a uint8 tensor of moe_mxfp8_packed_scale_bytes bytes."""
    s = _cuda(s, torch.uint8, "s")
    K = s.shape[-1] * 32
    rows = s.numel() // s.shape[-1]
    out = torch.empty(max(moe_mxfp8_packed_scale_bytes(rows, K), 16), dtype=torch.uint8, device=s.device)
    _check("moe_mxfp8_pack_scales", lib().moe_mxfp8_pack_scales(_ptr(s), rows, K, _ptr(out), _stream("s", s)))
    return out


def moe_fp8_block_pack_weights(w):
    """e4m3 expert weights [E, N, K] -> the tile-packed layout, a uint8 tensor of shape
    [E, N/128, K/128, 128, 128] (each 128x128 block contiguous; load-time, once)."""
    w = _codes(_cuda(w, None, "w"))
    E, N, K = w.shape
    packed = torch.empty(E, N // 128, K // 128, 128, 128, dtype=torch.uint8, device=w.device)
    _check("moe_fp8_block_pack_weights",
           lib().moe_fp8_block_pack_weights(_ptr(w), E, N, K, _ptr(packed), _stream("w", w)))
    return packed


def moe_nvfp4_quant_weight(w):
    """NVFP4 quantisation of bf16 expert weights [E, N, K] (page "vllm.model_executor.layers.
    quantization.online.nvfp4", _quantize_moe_weight_to_nvfp4): returns (codes uint8 [E, N, K/2],
    two e2m1 per byte, element 2i in the low nibble; block scales uint8 [E, N, K/16], e4m3 bits;
    global scales fp32 [E], the factor that dequantises)."""
    _cuda(w, torch.bfloat16, "w")
    E, N, K = w.shape
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device)
    sf = torch.empty(E, N, K // 16, dtype=torch.uint8, device=w.device)
    gs = torch.empty(E, dtype=torch.float32, device=w.device)
    _check("moe_nvfp4_quant_weight",
           lib().moe_nvfp4_quant_weight(_ptr(w), E, N, K, _ptr(q), _ptr(sf), _ptr(gs), _stream("w", w)))
    return q, sf, gs


def moe_nvfp4_pack_weights(q, block_scale):
    """NVFP4 codes [E, N, K/2] and block scales [E, N, K/16] -> the packed layout the forward
    reads (MOE_WEIGHTS_NVFP4): uint8 [E, N/16, K/128, 1152] (load-time, once)."""
    q = _cuda(q, torch.uint8, "q")
    block_scale = _codes(_cuda(block_scale, None, "block_scale"))
    E, N, K2 = q.shape
    K = 2 * K2
    if block_scale.shape != (E, N, K // 16):
        raise ValueError("block_scale must be [E, N, K/16]")
    packed = torch.empty(E, N // 16, K // 128, NVFP4_UNIT_BYTES, dtype=torch.uint8, device=q.device)
    _check("moe_nvfp4_pack_weights",
           lib().moe_nvfp4_pack_weights(_ptr(q), _ptr(block_scale), E, N, K, _ptr(packed),
                                        _stream("q block_scale", q, block_scale)))
    return packed


def moe_nvfp4_packed_bytes(E, N, K) -> int:
    return int(lib().moe_nvfp4_packed_bytes(E, N, K))


def _weight_shape(w):
    """(E, N, K, layout) of expert weights in any of the layouts."""
    if w.dim() == 5:
        return w.shape[0], w.shape[1] * 128, w.shape[2] * 128, MOE_WEIGHTS_TILED
    if w.dim() == 4 and w.shape[3] == NVFP4_UNIT_BYTES:
        return w.shape[0], w.shape[1] * 16, w.shape[2] * 128, MOE_WEIGHTS_NVFP4
    E, N, K = w.shape
    return E, N, K, MOE_WEIGHTS_NK


def fp8_block_grouped_gemm(A, a_scale, a_scale_strides, B, b_scale, tile_expert, tile_row0, num_tiles,
                           epilogue="store", out_f32=None, out_q=None, out_scale=None, out_scale_strides=(0, 0),
                           sorted_pair_ids=None, topk_weights=None, topk=1, num_pairs=0, out_bf16=None,
                           scale_fmt="f32"):
    """Grouped GEMM of the C ABI.  Outputs are caller-provided tensors (see include/moefp8.h)."""
    A, B = _codes(_cuda(A, None, "A")), _codes(_cuda(B, None, "B"))
    E, N, K, layout = _weight_shape(B)
    ep = _Epilogue(EPILOGUE[epilogue], topk, _ptr(out_f32), _ptr(out_q), _ptr(out_scale),
                   int(out_scale_strides[0]), int(out_scale_strides[1]), _ptr(sorted_pair_ids),
                   _ptr(topk_weights), int(num_pairs), _ptr(out_bf16), layout, SCALE_FMT[scale_fmt])
    rc = lib().fp8_block_grouped_gemm(_ptr(A), _ptr(a_scale), int(a_scale_strides[0]), int(a_scale_strides[1]),
                                      A.shape[0], _ptr(B), _ptr(b_scale), N, K, E, _ptr(tile_expert),
                                      _ptr(tile_row0), _ptr(num_tiles), tile_expert.numel(), ctypes.byref(ep),
                                      _stream("A B", A, B))
    _check("fp8_block_grouped_gemm", rc)


def moe_unpermute_sum(y, pos, T, topk, out=None):
    """out[t] = bf16(sum_j y[pos[t*topk + j]]) for y fp32 [rows, H] and pos int32 [T*topk]."""
    _cuda(y, torch.float32, "y")
    _cuda(pos, torch.int32, "pos")
    H = y.shape[1]
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    rc = lib().moe_unpermute_sum(_ptr(y), y.shape[0], _ptr(pos), T, topk, H, _ptr(out), _stream("y pos", y, pos))
    _check("moe_unpermute_sum", rc)
    return out


def moe_combine_pairs(y, pos, T, topk, out=None):
    """out[t] = bf16(sum_j y[t*topk + j]) over pairs with pos >= 0, for y bf16 [T*topk, H] in pair order."""
    _cuda(y, torch.bfloat16, "y")
    _cuda(pos, torch.int32, "pos")
    H = y.shape[1]
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    rc = lib().moe_combine_pairs(_ptr(y), _ptr(pos), T, topk, H, _ptr(out), _stream("y pos", y, pos))
    _check("moe_combine_pairs", rc)
    return out


def moe_fp8_block_pair_path(T, H, E, topk, scale_fmt="f32") -> int:
    """Two-CTA clusters that the step's tile GEMMs launch on the CTA-pair kernel (0: the one-CTA
    kernels)."""
    r = int(lib().moe_fp8_block_pair_path(T, H, E, topk, SCALE_FMT[scale_fmt]))
    if r < 0:
        raise MoeError("moe_fp8_block_pair_path", r)
    return r


def moe_fp8_block_decode_path(T, H, I, topk, decode="auto") -> bool:
    """Whether a step of T tokens takes the decode-path GEMMs under `decode` (auto / off / on)."""
    r = int(lib().moe_fp8_block_decode_path(T, H, I, topk, DECODE_PATH[decode]))
    if r < 0:
        raise ValueError(f"moe_fp8_block_decode_path({T}, {H}, {I}, {topk}, {decode!r})")
    return bool(r)


def moe_fp8_block_forward_kernel_count(T, H, I, E, topk, routing: RoutingParams | None = None, layout=None,
                                       scale_fmt="f32", decode="auto") -> int:
    """Kernels one moe_fp8_block_forward with these routing parameters and options launches
    (layout: MOE_WEIGHTS_NK / _TILED / _NVFP4, default NK)."""
    if routing is None and layout is None and scale_fmt == "f32" and decode == "auto":
        return int(lib().moe_fp8_block_forward_kernel_count(T, H, I, E, topk))
    rp = routing.to_c() if routing else None
    opts = _ForwardOptions(MOE_WEIGHTS_NK if layout is None else layout, SCALE_FMT[scale_fmt], DECODE_PATH[decode])
    return int(lib().moe_fp8_block_forward_kernel_count_ex(T, H, I, E, topk, ctypes.byref(rp) if rp else None,
                                                           ctypes.byref(opts)))


def moe_fp8_block_workspace_size(T, H, I, E, topk) -> int:
    return int(lib().moe_fp8_block_workspace_size(T, H, I, E, topk))


_ws_cache: dict = {}


def _workspace(device, nbytes):
    key = (device.type, device.index)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


FORWARD_STAGES = ("route", "sort", "quant", "gemm_w13", "gemm_w2", "unpermute_sum")


def moe_fp8_block_forward(hidden, router_logits, w13, w13_scale, w2, w2_scale, topk, renormalize=True,
                          routing: RoutingParams | None = None, out=None, workspace=None, events=None,
                          scale_fmt="f32", decode="auto"):
    """The whole layer: returns bf16 [T, H] (written into `out` when given).

    w13 / w2 in the pages' layout [E, N, K] or tile-packed (moe_fp8_block_pack_weights, 5-D), or
    NVFP4-packed (moe_nvfp4_pack_weights, 4-D) with w13_scale / w2_scale the global scales [E].
    scale_fmt "ue8m0_packed": w13_scale / w2_scale are moe_fp8_block_pack_scales outputs and both
    GEMMs run on the block-scaled MMA.
    decode: "auto", "off" or "on" -- the decode-path GEMMs for small steps (MOE_DECODE_*).
    events: optional list of 7 torch.cuda.Event recorded between the stages
    (FORWARD_STAGES) on the current stream, for per-stage timing."""
    _cuda(hidden, torch.bfloat16, "hidden")
    _cuda(router_logits, torch.float32, "router_logits")
    w13, w2 = _codes(_cuda(w13, None, "w13")), _codes(_cuda(w2, None, "w2"))
    sdt = torch.uint8 if scale_fmt in _PACKED_SCALES else torch.float32
    _cuda(w13_scale, sdt, "w13_scale")
    _cuda(w2_scale, sdt, "w2_scale")
    T, H = hidden.shape
    E, N1, _, layout = _weight_shape(w13)
    if _weight_shape(w2)[3] != layout:
        raise ValueError("w13 and w2 must share one layout")
    I = N1 // 2
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=hidden.device)
    nbytes = moe_fp8_block_workspace_size(T, H, I, E, topk)
    if workspace is None:
        workspace = _workspace(hidden.device, nbytes)
    rp = routing.to_c() if routing else None
    opts = _ForwardOptions(layout, SCALE_FMT[scale_fmt], DECODE_PATH[decode])
    arr = None
    if events is not None:
        if len(events) != len(FORWARD_STAGES) + 1:
            raise ValueError("events: one more than the number of stages")
        for ev in events:
            if not ev.cuda_event:       # torch creates the CUDA event on its first record()
                ev.record()
        arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(ev.cuda_event) for ev in events])
    rc = lib().moe_fp8_block_forward_ex(_ptr(hidden), _ptr(router_logits), _ptr(w13), _ptr(w13_scale), _ptr(w2),
                                        _ptr(w2_scale), T, H, I, E, topk, int(bool(renormalize)),
                                        ctypes.byref(rp) if rp else None, ctypes.byref(opts), _ptr(workspace),
                                        workspace.numel(), _ptr(out),
                                        _stream("hidden router_logits w13 w13_scale w2 w2_scale", hidden,
                                                router_logits, w13, w13_scale, w2, w2_scale), arr)
    _check("moe_fp8_block_forward", rc)
    return out


def moe_nvfp4_forward(hidden, router_logits, w13, w13_global_scale, w2, w2_global_scale, topk, renormalize=True,
                      routing: RoutingParams | None = None, out=None, workspace=None, events=None, scale_fmt="f32"):
    """The layer on NVFP4 expert weights (moe_nvfp4_pack_weights outputs and their global scales
    [E]); activations and the intermediate in FP8 1x128 groups (scale_fmt)."""
    if _weight_shape(w13)[3] != MOE_WEIGHTS_NVFP4 or _weight_shape(w2)[3] != MOE_WEIGHTS_NVFP4:
        raise ValueError("w13 and w2 must be NVFP4-packed (moe_nvfp4_pack_weights)")
    return moe_fp8_block_forward(hidden, router_logits, w13, w13_global_scale, w2, w2_global_scale, topk,
                                 renormalize, routing, out, workspace, events, scale_fmt, "on")


def moe_fp8_block_masked_workspace_size(E, max_tokens, H, I) -> int:
    return int(lib().moe_fp8_block_masked_workspace_size(E, max_tokens, H, I))


def moe_fp8_block_forward_masked(hidden, counts, w13, w13_scale, w2, w2_scale, out=None, workspace=None,
                                 scale_fmt="f32"):
    """Expert MLP on the masked batched layout: hidden bf16 [E, M, H] with counts int32 [E]
    (CUDA) valid rows per expert; returns bf16 [E, M, H] (rows past the counts not written)."""
    _cuda(hidden, torch.bfloat16, "hidden")
    _cuda(counts, torch.int32, "counts")
    w13, w2 = _codes(_cuda(w13, None, "w13")), _codes(_cuda(w2, None, "w2"))
    sdt = torch.uint8 if scale_fmt in _PACKED_SCALES else torch.float32
    _cuda(w13_scale, sdt, "w13_scale")
    _cuda(w2_scale, sdt, "w2_scale")
    E, M, H = hidden.shape
    _, N1, _, layout = _weight_shape(w13)
    if _weight_shape(w2)[3] != layout:
        raise ValueError("w13 and w2 must share one layout")
    I = N1 // 2
    if out is None:
        out = torch.empty(E, M, H, dtype=torch.bfloat16, device=hidden.device)
    nbytes = moe_fp8_block_masked_workspace_size(E, M, H, I)
    if workspace is None:
        workspace = _workspace(hidden.device, nbytes)
    rc = lib().moe_fp8_block_forward_masked(_ptr(hidden), _ptr(counts), _ptr(w13), _ptr(w13_scale), _ptr(w2),
                                            _ptr(w2_scale), E, M, H, I, ctypes.byref(_ForwardOptions(layout,
                                            SCALE_FMT[scale_fmt], 0)), _ptr(workspace), workspace.numel(),
                                            _ptr(out), _stream("hidden counts w13 w13_scale w2 w2_scale", hidden,
                                                               counts, w13, w13_scale, w2, w2_scale))
    _check("moe_fp8_block_forward_masked", rc)
    return out


# ---- training operators (C ABI section "training") ------------------------------------------
# They record nothing for autograd: results have no grad_fn, and the gradients are the functions named
# *_backward, *_dgrad and *_wgrad, which the caller runs.

DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

try:   # half the time of torch.empty, which counts in a step of one token
    _empty_strided = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:
    def _empty_strided(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _training_stream(function, names, *operands, stacklevel=3):
    """_stream of a training operator, with a warning where autograd would have recorded it."""
    device = _device()
    for t in operands:
        if t is not None and (t.requires_grad or t.get_device() != device):
            stream = _stream(names, *operands)
            if torch.is_grad_enabled():
                warnings.warn(f"{function} records nothing for autograd, so no gradient reaches its operands through "
                              "backward(): run the gradient functions, and this one under torch.no_grad()",
                              stacklevel=stacklevel)
            return stream
    return _raw_stream(device)


def _vector(n, dtype):
    """A new [n] on the current device, where the kernels run."""
    return _empty_strided((n,), (1,), dtype)


def _matrix(n, m, dtype):
    return _empty_strided((n, m), (m, 1), dtype)


_INT_MAX = 2 ** 31 - 1   # sizes are C ints, to which ctypes cuts without a word


def _too_large(name):
    return ValueError(f"{name} has a size past 2^31 - 1")


def _typed(t, name, like=None):
    """Code of t's element type; with `like`, t must have that tensor's type."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    code = DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _rows(t, name, like=None, shape=None):
    """A matrix whose columns are adjacent: (type code, row stride)."""
    code = _typed(t, name, like)
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be {list(shape) if shape is not None else 'a matrix'}, got {list(t.shape)}")
    n, cols = t.shape
    if n > _INT_MAX or cols > _INT_MAX:
        raise _too_large(name)
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name} must have adjacent columns")
    if n <= 1:
        return code, cols
    if s0 < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    return code, s0


def _dense(t, name, dtype, shape):
    _cuda(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


@dataclasses.dataclass
class Dispatch:
    """Token rows sorted by expert (moe_dispatch)."""
    rows: torch.Tensor             # [T*topk, H]; rows of no pair are zero
    expert_offsets: torch.Tensor   # int32 [E+1]
    pair_ids: torch.Tensor         # int32 [T*topk], -1 for a row of no pair
    pos: torch.Tensor              # int32 [T, topk], -1 for a dropped pair


def moe_dispatch(x, topk_ids, num_experts) -> Dispatch:
    """Rows of x [T, H] (bf16, fp16 or fp32) sorted by expert: rows[pos[t, j]] = x[t], the pairs of an
    expert in ascending order, nothing padded.  topk_ids int32 [T, topk]; a negative id drops its pair."""
    code, ld = _rows(x, "x")
    _cuda(topk_ids, torch.int32, "topk_ids")
    T, H = x.shape
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError(f"topk_ids must be [{T}, topk], got {list(topk_ids.shape)}")
    k = topk_ids.shape[1]
    if k > _INT_MAX:
        raise _too_large("topk_ids")
    if abs(num_experts) > _INT_MAX:
        raise ValueError(f"num_experts must be an int below 2^31, got {num_experts}")
    P = T * k
    L = lib()
    wsb = L.moe_dispatch_workspace_size(T, k, num_experts)
    stream = _training_stream("moe_dispatch", "x topk_ids", x, topk_ids)
    ws = _vector(wsb, torch.uint8) if wsb else None
    rows = _matrix(P, H, x.dtype)
    offsets = _vector(max(num_experts, 0) + 1, torch.int32)
    pair_ids = _vector(P, torch.int32)
    pos = _matrix(T, k, torch.int32)
    rc = L.moe_dispatch(x.data_ptr(), ld, code, topk_ids.data_ptr(), T, k, num_experts, H, rows.data_ptr(),
                        offsets.data_ptr(), pair_ids.data_ptr(), pos.data_ptr(), None if ws is None else ws.data_ptr(),
                        wsb, stream)
    _check("moe_dispatch", rc)
    return Dispatch(rows, offsets, pair_ids, pos)


def _pos(pos):
    _cuda(pos, torch.int32, "pos")
    if pos.dim() != 2:
        raise ValueError(f"pos must be [T, topk], got {list(pos.shape)}")
    T, k = pos.shape
    if T > _INT_MAX or k > _INT_MAX:
        raise _too_large("pos")
    return T, k


def moe_dispatch_backward(drows, pos):
    """Gradient of x: dx[t] = sum_j drows[pos[t, j]], [T, H] in drows' type."""
    code, ld = _rows(drows, "drows")
    T, k = _pos(pos)
    n, H = drows.shape
    stream = _training_stream("moe_dispatch_backward", "drows pos", drows, pos)
    dx = _matrix(T, H, drows.dtype)
    _check("moe_dispatch_backward", lib().moe_dispatch_backward(drows.data_ptr(), ld, code, pos.data_ptr(), T, k, H, n,
                                                                dx.data_ptr(), stream))
    return dx


def moe_combine(y, pos, weights=None):
    """The experts' rows back to their tokens: out[t] = sum_j weights[t, j] * y[pos[t, j]] over the
    pairs with a row (weights fp32 [T, topk]; None: 1), [T, H] in y's type."""
    code, ld = _rows(y, "y")
    T, k = _pos(pos)
    if weights is not None:
        _dense(weights, "weights", torch.float32, (T, k))
    n, H = y.shape
    stream = _training_stream("moe_combine", "y pos weights", y, pos, weights)
    out = _matrix(T, H, y.dtype)
    _check("moe_combine", lib().moe_combine(y.data_ptr(), ld, code, pos.data_ptr(),
                                            None if weights is None else weights.data_ptr(), T, k, H, n,
                                            out.data_ptr(), stream))
    return out


def moe_combine_backward(dout, y, pos, pair_ids, weights=None):
    """Gradients of moe_combine: (dy [rows, H] in y's type, zero in rows of no pair; dweights fp32 [T, topk])."""
    code, ldy = _rows(y, "y")
    T, k = _pos(pos)
    n, H = y.shape
    _, ldo = _rows(dout, "dout", y, (T, H))
    _dense(pair_ids, "pair_ids", torch.int32, (n,))
    if weights is not None:
        _dense(weights, "weights", torch.float32, (T, k))
    stream = _training_stream("moe_combine_backward", "dout y pos pair_ids weights", dout, y, pos, pair_ids, weights)
    dy = _matrix(n, H, y.dtype)
    dw = _matrix(T, k, torch.float32)
    rc = lib().moe_combine_backward(dout.data_ptr(), ldo, y.data_ptr(), ldy, code, pos.data_ptr(), pair_ids.data_ptr(),
                                    None if weights is None else weights.data_ptr(), T, k, H, n, dy.data_ptr(),
                                    dw.data_ptr(), stream)
    _check("moe_combine_backward", rc)
    return dy, dw


GATE_KIND = {"none": 0, "token": 1, "channel": 2, "full": 3}


class _PostNormParams(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("next_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_stride", ctypes.c_int64), ("weight_dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("gate_sigmoid", ctypes.c_int32), ("weight_offset", ctypes.c_float), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float)]


def _norm_weight(w, H, name):
    code = _typed(w, name)
    if w.dim() != 1 or w.shape[0] != H or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{H}], got {list(w.shape)}")
    return code


def moe_pre_norm(x, weight, eps=1e-6, weight_offset=0.0):
    """RMS norm before a block: h = x * rstd * (weight + weight_offset).  Returns (h in x's type,
    rstd fp32 [T])."""
    code, ld = _rows(x, "x")
    T, H = x.shape
    wcode = _norm_weight(weight, H, "weight")
    stream = _training_stream("moe_pre_norm", "x weight", x, weight)
    h = _matrix(T, H, x.dtype)
    rstd = _vector(T, torch.float32)
    _check("moe_pre_norm", lib().moe_pre_norm(x.data_ptr(), ld, code, weight.data_ptr(), wcode, weight_offset, eps, T,
                                              H, h.data_ptr(), rstd.data_ptr(), stream))
    return h, rstd


def _norm_workspace(T, H):
    """Scratch of a norm's gradient and its size in bytes."""
    wsb = lib().moe_norm_backward_workspace_size(T, H)
    return _vector(wsb, torch.uint8), wsb


def moe_pre_norm_backward(dh, x, weight, rstd, dresidual=None, weight_offset=0.0):
    """Gradients of moe_pre_norm: (dx in x's type, dresidual included; dweight fp32 [H])."""
    code, ldx = _rows(x, "x")
    T, H = x.shape
    _, ldd = _rows(dh, "dh", x, (T, H))
    wcode = _norm_weight(weight, H, "weight")
    _dense(rstd, "rstd", torch.float32, (T,))
    dres, ldr = None, 0
    if dresidual is not None:
        _, ldr = _rows(dresidual, "dresidual", x, (T, H))
        dres = dresidual.data_ptr()
    stream = _training_stream("moe_pre_norm_backward", "dh x weight rstd dresidual", dh, x, weight, rstd, dresidual)
    dx = _matrix(T, H, x.dtype)
    dw = _vector(H, torch.float32)
    ws, wsb = _norm_workspace(T, H)
    rc = lib().moe_pre_norm_backward(dh.data_ptr(), ldd, x.data_ptr(), ldx, code, weight.data_ptr(), wcode, weight_offset,
                                     rstd.data_ptr(), dres, ldr, T, H, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), wsb,
                                     stream)
    _check("moe_pre_norm_backward", rc)
    return dx, dw


@dataclasses.dataclass
class PostNorm:
    """moe_post_norm: out and rstd, and the next block's norm of out (or None)."""
    out: torch.Tensor
    rstd: torch.Tensor
    next_h: torch.Tensor | None = None
    next_rstd: torch.Tensor | None = None


@dataclasses.dataclass
class PostNormGrads:
    """moe_post_norm_backward: dresidual and dgate are None where not wanted."""
    dy: torch.Tensor
    dweight: torch.Tensor               # fp32 [H]
    dresidual: torch.Tensor | None = None
    dgate: torch.Tensor | None = None   # token, full: the gate's type and shape; channel: fp32 [H]


def _post_norm_params(y, weight, gate, gate_kind, gate_sigmoid, residual_scale, block_scale, eps, weight_offset,
                      next_weight=None):
    T, H = y.shape
    wcode = _norm_weight(weight, H, "weight")
    if next_weight is not None and _norm_weight(next_weight, H, "next_weight") != wcode:
        raise TypeError("next_weight must have weight's type")
    if gate_kind not in GATE_KIND:
        raise ValueError(f"gate_kind must be one of {list(GATE_KIND)}, got {gate_kind!r}")
    if (gate is None) != (gate_kind == "none"):
        raise ValueError(f"gate_kind {gate_kind!r} and gate do not go together")
    gp, gs = None, 0
    if gate is not None:
        _typed(gate, "gate", y)
        if gate_kind == "full":
            _, gs = _rows(gate, "gate", y, (T, H))
        else:
            n = T if gate_kind == "token" else H
            if tuple(gate.shape) not in ((n,), (n, 1) if gate_kind == "token" else (1, n)):
                raise ValueError(f"a {gate_kind} gate must hold {n} values, got {list(gate.shape)}")
            gs = gate.stride(0 if gate_kind == "token" else -1) if n > 1 else 1
            if gs < 1 or (gate_kind == "channel" and gs != 1):
                raise ValueError(f"a {gate_kind} gate must not be broadcast"
                                 + (" or strided" if gate_kind == "channel" else ""))
        gp = gate.data_ptr()
    return _PostNormParams(weight.data_ptr(), None if next_weight is None else next_weight.data_ptr(), gp, gs, wcode,
                           GATE_KIND[gate_kind], int(bool(gate_sigmoid)), weight_offset, eps, residual_scale,
                           block_scale)


def moe_post_norm(y, residual, weight, gate=None, gate_kind="none", gate_sigmoid=False, residual_scale=1.0,
                  block_scale=1.0, eps=1e-6, weight_offset=0.0, next_weight=None) -> PostNorm:
    """RMS norm after a block with its gate and residual:
    out = residual_scale * residual + block_scale * g * (y * rstd * (weight + weight_offset)), g the gate
    (gate_kind "token": [T] or [T, 1], "channel": [H] or [1, H], "full": [T, H], in y's type) or its sigmoid.
    next_weight: also the next block's norm of out, as stored."""
    code, ldy = _rows(y, "y")
    T, H = y.shape
    _, ldr = _rows(residual, "residual", y, (T, H))
    prm = _post_norm_params(y, weight, gate, gate_kind, gate_sigmoid, residual_scale, block_scale, eps, weight_offset,
                            next_weight)
    stream = _training_stream("moe_post_norm", "y residual weight gate next_weight", y, residual, weight, gate, next_weight)
    r = PostNorm(_matrix(T, H, y.dtype),
                 _vector(T, torch.float32))
    h2 = r2 = None
    if next_weight is not None:
        r.next_h, r.next_rstd = _matrix(T, H, y.dtype), _vector(T, torch.float32)
        h2, r2 = r.next_h.data_ptr(), r.next_rstd.data_ptr()
    _check("moe_post_norm", lib().moe_post_norm(y.data_ptr(), ldy, residual.data_ptr(), ldr, code, ctypes.byref(prm), T,
                                                H, r.out.data_ptr(), r.rstd.data_ptr(), h2, r2, stream))
    return r


def moe_post_norm_backward(dout, y, weight, rstd, gate=None, gate_kind="none", gate_sigmoid=False,
                           residual_scale=1.0, block_scale=1.0, weight_offset=0.0, residual_grad=True) -> PostNormGrads:
    """Gradients of moe_post_norm for dout (with a next_weight: the gradient of out, the part that
    next_h sends there included).  residual_grad=False: dresidual = residual_scale * dout is not written."""
    code, ldy = _rows(y, "y")
    T, H = y.shape
    _, ldo = _rows(dout, "dout", y, (T, H))
    _dense(rstd, "rstd", torch.float32, (T,))
    prm = _post_norm_params(y, weight, gate, gate_kind, gate_sigmoid, residual_scale, block_scale, 0.0, weight_offset)
    stream = _training_stream("moe_post_norm_backward", "dout y weight rstd gate", dout, y, weight, rstd, gate)
    dy = _matrix(T, H, y.dtype)
    dres = _matrix(T, H, y.dtype) if residual_grad else None
    dw = _vector(H, torch.float32)
    dg = None
    if gate is not None:
        dg = torch.empty(gate.shape, dtype=torch.float32 if gate_kind == "channel" else gate.dtype, device=gate.device)
    ws, wsb = _norm_workspace(T, H)
    rc = lib().moe_post_norm_backward(dout.data_ptr(), ldo, y.data_ptr(), ldy, code, ctypes.byref(prm),
                                      rstd.data_ptr(), T, H, dy.data_ptr(), None if dres is None else dres.data_ptr(),
                                      None if dg is None else dg.data_ptr(), dw.data_ptr(), ws.data_ptr(), wsb, stream)
    _check("moe_post_norm_backward", rc)
    return PostNormGrads(dy, dw, dres, dg)


def _expert_operands(t, E, offsets, name):
    code, ld = _rows(t, name)
    if t.dtype == torch.float32:
        raise TypeError(f"{name} must be bfloat16 or float16")
    _dense(offsets, "expert_offsets", torch.int32, (E + 1,))
    return code, ld


def _expert_weights(w, like):
    if w.dim() != 3:
        raise ValueError(f"w must be [E, N, K], got {list(w.shape)}")
    _cuda(w, like.dtype, "w")
    E, N, K = w.shape
    if max(E, N, K) > _INT_MAX:
        raise _too_large("w")
    return E, N, K


def _expert_gemm(a, w, expert_offsets, epilogue, save_gate_up=False):
    E, N, K = _expert_weights(w, a)
    code, ld = _expert_operands(a, E, expert_offsets, "a")
    if a.shape[1] != K:
        raise ValueError(f"a must have {K} columns, got {a.shape[1]}")
    stream = _training_stream("moe_expert_gemm_silu_mul" if epilogue else "moe_expert_gemm", "a w expert_offsets", a, w,
                              expert_offsets, stacklevel=4)
    out = _matrix(a.shape[0], N // 2 if epilogue else N, a.dtype)
    gate_up = _matrix(a.shape[0], N, a.dtype) if save_gate_up else None
    rc = lib().moe_expert_gemm(a.data_ptr(), ld, code, w.data_ptr(), expert_offsets.data_ptr(), a.shape[0], E, N, K,
                               epilogue, out.data_ptr(), None if gate_up is None else gate_up.data_ptr(), stream)
    _check("moe_expert_gemm", rc)
    return out, gate_up


def moe_expert_gemm(a, w, expert_offsets):
    """The experts' product over rows sorted by expert: out[r] = a[r] @ w[e]^T for the rows
    [expert_offsets[e], expert_offsets[e+1]) of a [rows, K]; w [E, N, K]; bf16 or fp16.  Rows of no expert are zero."""
    return _expert_gemm(a, w, expert_offsets, 0)[0]


def moe_expert_gemm_silu_mul(a, w, expert_offsets, save_gate_up=True):
    """The first product with its activation: (h [rows, N/2] = silu(gate) * up, gate_up [rows, N] = the
    product itself, which the gradient needs; None with save_gate_up=False).  w [E, N, K]: gate rows, then up."""
    return _expert_gemm(a, w, expert_offsets, 1, save_gate_up)


def moe_expert_gemm_dgrad(dc, w, expert_offsets, gate_up=None):
    """The rows' gradient da[r] = dc[r] @ w[e], [rows, K]; with gate_up [rows, 2K], where a was
    silu(gate) * up, the gradient of gate_up instead."""
    E, N, K = _expert_weights(w, dc)
    code, ld = _expert_operands(dc, E, expert_offsets, "dc")
    n = dc.shape[0]
    if dc.shape[1] != N:
        raise ValueError(f"dc must have {N} columns, got {dc.shape[1]}")
    gp, ldgu = None, 0
    if gate_up is not None:
        _, ldgu = _rows(gate_up, "gate_up", dc, (n, 2 * K))
        gp = gate_up.data_ptr()
    stream = _training_stream("moe_expert_gemm_dgrad", "dc w expert_offsets gate_up", dc, w, expert_offsets, gate_up)
    out = _matrix(n, K if gate_up is None else 2 * K, dc.dtype)
    rc = lib().moe_expert_gemm_dgrad(dc.data_ptr(), ld, code, w.data_ptr(), expert_offsets.data_ptr(), n, E, N, K, gp,
                                     ldgu, out.data_ptr(), stream)
    _check("moe_expert_gemm_dgrad", rc)
    return out


def moe_expert_gemm_wgrad(dc, a, expert_offsets):
    """The weights' gradient dw[e] = dc[rows of e]^T @ a[rows of e], [E, N, K] in dc's type (zero for
    an expert without rows)."""
    if expert_offsets.dim() != 1 or expert_offsets.shape[0] < 2:
        raise ValueError(f"expert_offsets must be [E+1], got {list(expert_offsets.shape)}")
    E = expert_offsets.shape[0] - 1
    code, ldd = _expert_operands(dc, E, expert_offsets, "dc")
    _, lda = _rows(a, "a", dc)
    if a.shape[0] != dc.shape[0]:
        raise ValueError("dc and a must have the same rows")
    n, N = dc.shape
    K = a.shape[1]
    stream = _training_stream("moe_expert_gemm_wgrad", "dc a expert_offsets", dc, a, expert_offsets)
    dw = _empty_strided((E, N, K), (N * K, K, 1), dc.dtype)
    rc = lib().moe_expert_gemm_wgrad(dc.data_ptr(), ldd, a.data_ptr(), lda, code, expert_offsets.data_ptr(), n, E, N, K,
                                     dw.data_ptr(), stream)
    _check("moe_expert_gemm_wgrad", rc)
    return dw


def moe_clip_grads(grads, max_norm, norm_type=2.0, eps=1e-6, out=None):
    """Global norm of a list of contiguous gradient tensors (bf16, fp16, fp32, in any mix) and their
    clipping by min(1, max_norm / (norm + eps)): in place, or into the list `out` (same shapes and
    types), none of which may share memory with another result or gradient.  norm_type 2 or inf.
    Returns the norm before clipping, fp32, on the device."""
    grads = list(grads)
    out = grads if out is None else list(out)
    kind = {2.0: 0, float("inf"): 1}.get(float(norm_type))
    if kind is None:
        raise ValueError(f"norm_type must be 2 or inf, got {norm_type}")
    if len(out) != len(grads):
        raise ValueError("out must hold one tensor per gradient")
    n = len(grads)
    device = _device() if n and grads[0].is_cuda else None
    codes = [DTYPE.get(g.dtype, -1) for g in grads]
    if n and (-1 in codes or {g.get_device() for g in grads} != {device} or not all([g.is_contiguous() for g in grads])):
        for i, g in enumerate(grads):
            _typed(g, f"grads[{i}]")
            _stream(f"grads[{i}]", g)
            if not g.is_contiguous():
                raise ValueError(f"grads[{i}] must be contiguous")
    outs = ptrs = [g.data_ptr() for g in grads]
    if out is not grads:
        outs = []
        for i, (g, o) in enumerate(zip(grads, out)):
            if o.dtype != g.dtype or o.shape != g.shape or o.get_device() != device or not o.is_contiguous():
                raise ValueError(f"out[{i}] must be a contiguous CUDA tensor like grads[{i}], on its device")
            outs.append(o.data_ptr())
    L = lib()
    wsb = L.moe_clip_grads_workspace_size(n)
    ws = _vector(wsb, torch.uint8)
    total = _empty_strided((), (), torch.float32)
    sizes = list(map(torch.Tensor.numel, grads))   # (half the time of as many method calls)
    table, kinds = array.array("q", ptrs + outs + sizes), array.array("i", codes)   # host arrays of the C call
    at = table.buffer_info()[0]
    rc = L.moe_clip_grads(at, at + 8 * n, at + 16 * n, kinds.buffer_info()[0], n, kind, float(max_norm), float(eps),
                          total.data_ptr(), ws.data_ptr(), wsb, _stream())
    _check("moe_clip_grads", rc)
    torch.autograd.graph.increment_version(out)   # autograd then knows what it may have saved of them as changed
    return total


def moe_selftest_bounded_wait(expire=True):
    """Make one pipeline wait expire (about 2 s, MOE_STATUS_WAIT_TIMEOUT) or complete at once;
    read the outcome with moe_get_device_status."""
    _check("moe_selftest_bounded_wait", lib().moe_selftest_bounded_wait(int(bool(expire)), _stream()))


def moe_get_device_status(clear=False) -> int:
    """Device status bits (synchronises the device)."""
    st = ctypes.c_uint32(0)
    _check("moe_get_device_status", lib().moe_get_device_status(ctypes.byref(st), int(bool(clear))))
    return st.value
