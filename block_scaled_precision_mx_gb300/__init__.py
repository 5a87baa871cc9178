"""GB300 (sm_103a) block-scaled quantization and GEMMs: MXFP8, MXFP4, NVFP4, DeepSeek FP8; and an
8-bit key/value cache with block scales and the attention over it.

Thin Python binding over the C ABI of ``libmxgb.so`` (declared in include/mx.h).
Every function here only marshals arguments: tensors are torch CUDA tensors
(device memory), the stream is torch's current stream unless one is given,
and every step of the computation runs in the library's CUDA kernels.  There
is no CPU fallback: if the library cannot be loaded, every call raises.

Entry points (same names as the C ABI):
  mx_quantize, mx_quantize_dual, mx_gemm, nvfp4_quantize, nvfp4_gemm, fp8_blockwise_gemm,
  mx_gemm_grouped, mx_gemm_mxout, mx_scales_from_fp32_blocks, nvfp4_quantize_ex, nvfp4_quantize_2d,
  nvfp4_quantize_grouped, nvfp4_gemm_grouped, nvfp4_gemm_grouped_ex, fp8_blockwise_gemm_grouped, mx_scale_bytes,
  nvfp4_workspace_bytes, mx_check, kv_block_tables, kv_cache_append, kv_attention, qk_norm_rope,
  qk_norm_rope_backward, kv_draft_trees, kv_tree_attention, kv_verify_drafts, kv_cache_compact.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from .build import LIB as _LIB_PATH

# enums (include/mx.h)
MX_OK, MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED, MX_ERR_CUDA, MX_ERR_TIMEOUT = range(5)
E4M3, E5M2, E2M1 = 0, 1, 2
SCALE_E8M0, SCALE_UE4M3, SCALE_FP32, SCALE_FP32_POW2 = 0, 1, 2, 3
ROWWISE, COLWISE, BOTH = 1, 2, 3
OUT_F32, OUT_BF16 = 0, 1
HALF_BF16, HALF_F16 = 0, 1

EXPORTS = (
    "mx_abi_version", "mx_status_string", "mx_quantize", "mx_gemm", "nvfp4_workspace_bytes",
    "nvfp4_quantize", "nvfp4_gemm", "fp8_blockwise_gemm", "mx_scale_bytes", "mx_check", "mx_num_sms",
    "nvfp4_quantize_noalloc", "mx_quantize_dual", "mx_scales_from_fp32_blocks", "nvfp4_quantize_ex",
    "nvfp4_quantize_2d", "mx_gemm_grouped", "mx_gemm_mxout", "mx_unswizzle_scales", "mx_swizzle_scales",
    "mx_selftest_wait_timeout", "mx_gemm_mxout_ex", "nvfp4_gemm_grouped", "nvfp4_quantize_grouped",
    "nvfp4_gemm_grouped_ex", "fp8_blockwise_gemm_grouped", "kv_block_tables", "kv_cache_append",
    "kv_attention_workspace_bytes", "kv_attention", "qk_norm_rope", "qk_norm_rope_workspace_bytes",
    "qk_norm_rope_backward", "kv_draft_trees", "kv_tree_attention", "kv_verify_drafts", "kv_cache_compact",
)


class MxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libmxgb.so (built by build.py / __graft_entry__.build()).  Raises if missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libmxgb.so not built ({_LIB_PATH}); run __graft_entry__.build()")
        lib = ctypes.CDLL(_LIB_PATH)
        i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
        fp = ctypes.POINTER(ctypes.c_float)
        sig = {
            "mx_abi_version": (i32, []),
            "mx_status_string": (ctypes.c_char_p, [i32]),
            "mx_quantize": (i32, [vp, i64, i64, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp]),
            "mx_gemm": (i32, [vp, vp, i32, vp, vp, i32, i64, i64, i64, vp, i32, i64, vp]),
            "nvfp4_workspace_bytes": (ctypes.c_size_t, [i64, i64]),
            "nvfp4_quantize": (i32, [vp, i64, i64, vp, vp, vp, vp, vp]),
            "nvfp4_gemm": (i32, [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, i32, i64, vp]),
            "fp8_blockwise_gemm": (i32, [vp, vp, vp, vp, i64, i64, i64, vp, i32, i64, vp]),
            "mx_scale_bytes": (ctypes.c_size_t, [i64, i64, i32, i32, i32]),
            "mx_check": (i32, [vp]),
            "mx_num_sms": (i32, []),
            "nvfp4_quantize_noalloc": (i32, [vp, i64, i64, vp, vp, vp, vp]),
            "mx_quantize_dual": (i32, [vp, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "mx_scales_from_fp32_blocks": (i32, [vp, i64, i64, i32, vp, vp]),
            "nvfp4_quantize_ex": (i32, [vp, i64, i64, i32, ctypes.c_uint32, vp, vp, vp, vp, vp, vp]),
            "nvfp4_quantize_2d": (i32, [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp]),
            "mx_gemm_grouped": (i32, [vp, vp, i32, vp, vp, i32, vp, i64, i64, i64, i64, vp, i32, i64, vp]),
            "mx_gemm_mxout": (i32, [vp, vp, i32, vp, vp, i32, i64, i64, i64, i32, vp, vp, i64, vp]),
            "mx_unswizzle_scales": (i32, [vp, i64, i64, vp, vp]),
            "mx_swizzle_scales": (i32, [vp, i64, i64, vp, vp]),
            "mx_selftest_wait_timeout": (i32, [i64, vp]),
            "nvfp4_gemm_grouped": (i32, [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, i64, vp]),
            "nvfp4_quantize_grouped": (i32, [vp, i64, i64, vp, i64, vp, vp, vp, vp, vp]),
            "nvfp4_gemm_grouped_ex": (i32, [vp, vp, vp, i32, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, i64, vp]),
            "fp8_blockwise_gemm_grouped": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, i64, vp]),
            "mx_gemm_mxout_ex": (i32, [vp, vp, i32, vp, vp, i32, i64, i64, i64, i32, i32, vp, vp, i64, vp, vp, i64,
                                       vp]),
            "kv_block_tables": (i32, [vp, i64, i64, vp, vp, vp, i64, vp, i32, i64, vp, vp, vp, vp, vp]),
            "kv_cache_append": (i32, [vp, vp, i32, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, i32, i64, i64, i32, i32,
                                      vp]),
            "kv_attention_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64, i64, i64, i32]),
            "kv_attention": (i32, [vp, i32, i64, i64, i64, i64, vp, vp, vp, vp, i32, i64, i64, i32, i32, vp, i64, vp, vp,
                                   i64, i64, ctypes.c_float, i32, i64, vp, vp, vp, vp]),
            "qk_norm_rope": (i32, [vp, vp, i32, i64, i64, i64, i32, i64, i64, i64, i64, vp, vp, i32, vp, i64, i32, vp,
                                   ctypes.c_float, i32, vp, vp, i64, i64, i64, i64, vp]),
            "qk_norm_rope_workspace_bytes": (ctypes.c_size_t, [i32]),
            "qk_norm_rope_backward": (i32, [vp, vp, vp, vp, i32, i64, i64, i64, i32, *[i64] * 8, vp, vp, i32, vp, i64, i32, vp,
                                            ctypes.c_float, i32, vp, vp, i64, i64, i64, i64, vp, vp, vp, vp]),
            "kv_draft_trees": (i32, [vp, i64, vp, vp, i64, i64, i64, vp, i64, vp, vp]),
            "kv_tree_attention": (i32, [vp, i32, i64, i64, i64, i64, vp, vp, vp, vp, i32, i64, i64, i32, i32, vp, i64, vp, vp,
                                        i64, i64, vp, i64, vp, ctypes.c_float, i64, vp, vp, vp, vp]),
            "kv_verify_drafts": (i32, [vp, i64, vp, i64, i64, vp, vp, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp]),
            "kv_cache_compact": (i32, [vp, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, vp, i32, i64, i64, i32, i32, vp, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().mx_status_string(status).decode()


def _check(status: int, where: str):
    if status != MX_OK:
        raise MxError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:   # the current stream's handle without building a Stream object
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _u8(n, device):
    return torch.empty(int(n), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ sizes
def mx_scale_bytes(rows: int, cols: int, block: int = 32, block_rows: int = 1, sfmt: int = SCALE_E8M0) -> int:
    return int(load().mx_scale_bytes(rows, cols, block, block_rows, sfmt))


def nvfp4_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().nvfp4_workspace_bytes(rows, cols))


# ------------------------------------------------------------------ quantizers
def mx_quantize(x: torch.Tensor, block: int = 32, block_rows: int = 1, elem: int = E4M3,
                sfmt: int = SCALE_E8M0, layout: int = BOTH, q_row=None, s_row=None, q_col=None,
                s_col=None, stream=None):
    """Block-quantize bf16 x[rows][cols] (see include/mx.h, mx_quantize).

    Returns (q_row, s_row, q_col, s_col); outputs not given are allocated (torch), copies not
    requested are None.  MX scales are returned as flat uint8 tensors in the GEMM layout;
    DeepSeek FP32 scales as float tensors ([cols/128][rows] for 1x128, [rows/128][cols/128]
    for 128x128)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    rows, cols = x.shape
    dev = x.device
    row, col = bool(layout & ROWWISE), bool(layout & COLWISE)
    if sfmt in (SCALE_FP32, SCALE_FP32_POW2):
        if row and q_row is None:
            q_row = torch.empty(rows, cols, dtype=torch.uint8, device=dev)
        if row and s_row is None:
            shape = (cols // 128, rows) if block_rows == 1 else (rows // 128, cols // 128)
            s_row = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        per_byte = 2 if elem == E2M1 else 1          # MXFP4 codes are packed two per byte
        if row and q_row is None:
            q_row = torch.empty(rows, cols // per_byte, dtype=torch.uint8, device=dev)
        if row and s_row is None:
            s_row = _u8(mx_scale_bytes(rows, cols, block, block_rows, sfmt), dev)
        if col and q_col is None:
            q_col = torch.empty(cols, rows // per_byte, dtype=torch.uint8, device=dev)
        if col and s_col is None:
            s_col = _u8(mx_scale_bytes(cols, rows, block, block_rows, sfmt), dev)
    st = load().mx_quantize(_ptr(x), rows, cols, block, block_rows, elem, sfmt, layout,
                            _ptr(q_row) if row else None, _ptr(s_row) if row else None,
                            _ptr(q_col) if col else None, _ptr(s_col) if col else None, _stream(stream))
    _check(st, "mx_quantize")
    return (q_row if row else None, s_row if row else None, q_col if col else None, s_col if col else None)


def mx_scales_from_fp32_blocks(s: torch.Tensor, rows: int, cols: int, block_rows: int, out=None, stream=None):
    """Per-32 E8M0 scales (MX GEMM layout, flat uint8) for a [rows][cols] code matrix from its
    power-of-two FP32 block scales (include/mx.h, mx_scales_from_fp32_blocks)."""
    if s.dtype != torch.float32:
        raise ValueError("s must be float32")
    if out is None:
        out = _u8(rows * cols // 32, s.device)
    st = load().mx_scales_from_fp32_blocks(_ptr(s), rows, cols, block_rows, _ptr(out), _stream(stream))
    _check(st, "mx_scales_from_fp32_blocks")
    return out


def mx_selftest_wait_timeout(budget_us: int = 10000, stream=None):
    """Make one device-side bounded wait run out (include/mx.h, mx_selftest_wait_timeout); the
    next mx_check() reports MX_ERR_TIMEOUT."""
    _check(load().mx_selftest_wait_timeout(budget_us, _stream(stream)), "mx_selftest_wait_timeout")


def mx_unswizzle_scales(s: torch.Tensor, rows: int, nblocks: int, out=None, stream=None):
    """GEMM-layout scale bytes -> plain uint8 [rows][nblocks] (include/mx.h, mx_unswizzle_scales);
    nblocks = K/32 for MX scales, K/16 for NVFP4 scales."""
    if s.dtype != torch.uint8:
        raise ValueError("s must be uint8")
    if out is None:
        out = torch.empty(rows, nblocks, dtype=torch.uint8, device=s.device)
    _check(load().mx_unswizzle_scales(_ptr(s), rows, nblocks, _ptr(out), _stream(stream)), "mx_unswizzle_scales")
    return out


def mx_swizzle_scales(plain: torch.Tensor, out=None, stream=None):
    """plain uint8 [rows][nblocks] -> GEMM-layout scale bytes, flat (include/mx.h, mx_swizzle_scales)."""
    if plain.dtype != torch.uint8 or plain.dim() != 2:
        raise ValueError("plain must be a 2-D uint8 tensor")
    rows, nblocks = plain.shape
    if out is None:
        out = _u8(rows * nblocks, plain.device)
    _check(load().mx_swizzle_scales(_ptr(plain), rows, nblocks, _ptr(out), _stream(stream)), "mx_swizzle_scales")
    return out


def mx_quantize_dual(x: torch.Tensor, layout: int = BOTH, e4m3=None, e5m2=None, stream=None):
    """E4M3 and E5M2 MX quantization of bf16 x from one read (include/mx.h, mx_quantize_dual).
    e4m3 / e5m2: optional (q_row, s_row, q_col, s_col) output tuples; returns both tuples."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    rows, cols = x.shape
    dev = x.device
    row, col = bool(layout & ROWWISE), bool(layout & COLWISE)

    def alloc():
        return (torch.empty(rows, cols, dtype=torch.uint8, device=dev) if row else None,
                _u8(mx_scale_bytes(rows, cols), dev) if row else None,
                torch.empty(cols, rows, dtype=torch.uint8, device=dev) if col else None,
                _u8(mx_scale_bytes(cols, rows), dev) if col else None)
    e4m3 = e4m3 if e4m3 is not None else alloc()
    e5m2 = e5m2 if e5m2 is not None else alloc()
    st = load().mx_quantize_dual(_ptr(x), rows, cols, layout, *[_ptr(t) for t in e4m3], *[_ptr(t) for t in e5m2],
                                 _stream(stream))
    _check(st, "mx_quantize_dual")
    return e4m3, e5m2


def nvfp4_quantize(x: torch.Tensor, q_packed=None, s_ue4m3=None, gscale=None, workspace=None, stream=None):
    """NVFP4 two-level quantization of bf16 x[rows][cols] (include/mx.h, nvfp4_quantize).
    Returns (q_packed [rows][cols/2] u8, s_ue4m3 flat u8 in the NVFP4 GEMM layout,
    gscale float[1])."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    rows, cols = x.shape
    dev = x.device
    if q_packed is None:
        q_packed = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    if s_ue4m3 is None:
        s_ue4m3 = _u8(mx_scale_bytes(rows, cols, 16, 1, SCALE_UE4M3), dev)
    if gscale is None:
        gscale = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _u8(max(16, nvfp4_workspace_bytes(rows, cols)), dev)
    st = load().nvfp4_quantize(_ptr(x), rows, cols, _ptr(q_packed), _ptr(s_ue4m3), _ptr(gscale),
                               _ptr(workspace), _stream(stream))
    _check(st, "nvfp4_quantize")
    return q_packed, s_ue4m3, gscale


def nvfp4_quantize_grouped(x: torch.Tensor, group_offsets: torch.Tensor, q_packed=None, s_ue4m3=None, gscale=None,
                           workspace=None, stream=None):
    """NVFP4 quantization of row groups of bf16 x[rows][cols], each group with its own global scale
    (include/mx.h, nvfp4_quantize_grouped).  group_offsets: int64 CUDA tensor [G + 1].  Returns
    (q_packed [rows][cols/2] u8, s_ue4m3 flat u8 in the NVFP4 GEMM layout, gscale float[G])."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    if group_offsets.dtype != torch.int64:
        raise ValueError("group_offsets must be int64")
    rows, cols = x.shape
    dev = x.device
    groups = group_offsets.numel() - 1
    if q_packed is None:
        q_packed = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    if s_ue4m3 is None:
        s_ue4m3 = _u8(mx_scale_bytes(rows, cols, 16, 1, SCALE_UE4M3), dev)
    if gscale is None:
        gscale = torch.empty(max(groups, 1), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _u8(max(16, (4 * groups + 15) // 16 * 16), dev)
    st = load().nvfp4_quantize_grouped(_ptr(x), rows, cols, _ptr(group_offsets), groups, _ptr(q_packed),
                                       _ptr(s_ue4m3), _ptr(gscale), _ptr(workspace), _stream(stream))
    _check(st, "nvfp4_quantize_grouped")
    return q_packed, s_ue4m3, gscale


def nvfp4_quantize_ex(x: torch.Tensor, rht: bool = False, signs: int = 0, rbits=None, q_packed=None,
                      s_ue4m3=None, gscale=None, workspace=None, stream=None):
    """NVFP4 with the 16-point random Hadamard transform (rht, 16-bit sign mask) and/or stochastic
    rounding (rbits: uint8 [rows][cols] random bytes) (include/mx.h, nvfp4_quantize_ex).
    Returns (q_packed, s_ue4m3, gscale) as nvfp4_quantize."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    rows, cols = x.shape
    dev = x.device
    if q_packed is None:
        q_packed = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    if s_ue4m3 is None:
        s_ue4m3 = _u8(mx_scale_bytes(rows, cols, 16, 1, SCALE_UE4M3), dev)
    if gscale is None:
        gscale = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _u8(max(16, nvfp4_workspace_bytes(rows, cols)), dev)
    st = load().nvfp4_quantize_ex(_ptr(x), rows, cols, int(bool(rht)), int(signs),
                                  None if rbits is None else _ptr(rbits), _ptr(q_packed), _ptr(s_ue4m3),
                                  _ptr(gscale), _ptr(workspace), _stream(stream))
    _check(st, "nvfp4_quantize_ex")
    return q_packed, s_ue4m3, gscale


def nvfp4_quantize_2d(x: torch.Tensor, out=None, gscale=None, workspace=None, stream=None):
    """NVFP4 with 16x16 blocks, both orientations (include/mx.h, nvfp4_quantize_2d).
    Returns (q_row, s_row, q_col, s_col, gscale)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    rows, cols = x.shape
    dev = x.device
    if out is None:
        out = (torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev),
               _u8(mx_scale_bytes(rows, cols, 16, 1, SCALE_UE4M3), dev),
               torch.empty(cols, rows // 2, dtype=torch.uint8, device=dev),
               _u8(mx_scale_bytes(cols, rows, 16, 1, SCALE_UE4M3), dev))
    if gscale is None:
        gscale = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _u8(max(16, nvfp4_workspace_bytes(rows, cols)), dev)
    st = load().nvfp4_quantize_2d(_ptr(x), rows, cols, *[_ptr(t) for t in out], _ptr(gscale), _ptr(workspace),
                                  _stream(stream))
    _check(st, "nvfp4_quantize_2d")
    return (*out, gscale)


# ------------------------------------------------------------------ GEMMs
def _out(M, N, out_dtype, out, dev):
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32, device=dev)
    return out, out.stride(0)


def mx_gemm(qa, sa, ea, qb, sb, eb, M, N, K, out_dtype=OUT_BF16, out=None, stream=None):
    """C[m][n] = sum_b sA sB sum_i qA qB (MXFP8, or MXFP4 with packed E2M1 codes; include/mx.h
    mx_gemm)."""
    out, ldc = _out(M, N, out_dtype, out, qa.device)
    st = load().mx_gemm(_ptr(qa), _ptr(sa), ea, _ptr(qb), _ptr(sb), eb, M, N, K, out.data_ptr(), out_dtype, ldc,
                        _stream(stream))
    _check(st, "mx_gemm")
    return out


def mx_gemm_mxout(qa, sa, ea, qb, sb, eb, M, N, K, out_elem=E4M3, q_out=None, s_out=None, stream=None):
    """MXFP8 GEMM with the MX quantization of its results fused into the epilogue (include/mx.h,
    mx_gemm_mxout).  Returns (q_out [M][N] u8 codes, s_out flat u8 scales in the MX GEMM layout)."""
    dev = qa.device
    if q_out is None:
        q_out = torch.empty(M, N, dtype=torch.uint8, device=dev)
    if s_out is None:
        s_out = _u8(M * N // 32, dev)
    st = load().mx_gemm_mxout(_ptr(qa), _ptr(sa), ea, _ptr(qb), _ptr(sb), eb, M, N, K, out_elem, _ptr(q_out),
                              _ptr(s_out), q_out.stride(0), _stream(stream))
    _check(st, "mx_gemm_mxout")
    return q_out, s_out


def nvfp4_gemm_grouped(qa, sa, ga, qb, sb, gb, group_offsets, M, N, K, out_dtype=OUT_F32, out=None, stream=None):
    """NVFP4 grouped GEMM (include/mx.h, nvfp4_gemm_grouped): rows off[g] .. off[g+1] of A times the
    g-th [N][K] block of B, scaled by ga * gb[g].  ga: float CUDA tensor [1]; gb: [G]."""
    if group_offsets.dtype != torch.int64:
        raise ValueError("group_offsets must be int64")
    out, ldc = _out(M, N, out_dtype, out, qa.device)
    st = load().nvfp4_gemm_grouped(_ptr(qa), _ptr(sa), _ptr(ga), _ptr(qb), _ptr(sb), _ptr(gb), _ptr(group_offsets),
                                   group_offsets.numel() - 1, M, N, K, out.data_ptr(), out_dtype, ldc,
                                   _stream(stream))
    _check(st, "nvfp4_gemm_grouped")
    return out


def nvfp4_gemm_grouped_ex(qa, sa, ga, ga_per_group, qb, sb, gb, group_offsets, M, N, K, out_dtype=OUT_F32, out=None,
                          stream=None):
    """nvfp4_gemm_grouped with one global scale of A per group when ga_per_group (ga: float CUDA
    tensor [G], e.g. from nvfp4_quantize_grouped over the same offsets) (include/mx.h)."""
    if group_offsets.dtype != torch.int64:
        raise ValueError("group_offsets must be int64")
    out, ldc = _out(M, N, out_dtype, out, qa.device)
    st = load().nvfp4_gemm_grouped_ex(_ptr(qa), _ptr(sa), _ptr(ga), int(bool(ga_per_group)), _ptr(qb), _ptr(sb),
                                      _ptr(gb), _ptr(group_offsets), group_offsets.numel() - 1, M, N, K,
                                      out.data_ptr(), out_dtype, ldc, _stream(stream))
    _check(st, "nvfp4_gemm_grouped_ex")
    return out


def mx_gemm_mxout_ex(qa, sa, ea, qb, sb, eb, M, N, K, out_elem=E4M3, layout=BOTH, q_row=None, s_row=None,
                     q_col=None, s_col=None, stream=None):
    """MXFP8 GEMM with row-wise and / or column-wise MX quantization of its results in the epilogue
    (include/mx.h, mx_gemm_mxout_ex).  Returns (q_row [M][N], s_row, q_col [N][M], s_col); copies
    not requested are None; scales are flat uint8 in the MX GEMM layout."""
    dev = qa.device
    row, col = bool(layout & ROWWISE), bool(layout & COLWISE)
    if row and q_row is None:
        q_row = torch.empty(M, N, dtype=torch.uint8, device=dev)
    if row and s_row is None:
        s_row = _u8(M * N // 32, dev)
    if col and q_col is None:
        q_col = torch.empty(N, M, dtype=torch.uint8, device=dev)
    if col and s_col is None:
        s_col = _u8(M * N // 32, dev)
    if not row:
        q_row = s_row = None
    if not col:
        q_col = s_col = None
    st = load().mx_gemm_mxout_ex(_ptr(qa), _ptr(sa), ea, _ptr(qb), _ptr(sb), eb, M, N, K, out_elem, layout,
                                 _ptr(q_row), _ptr(s_row), N, _ptr(q_col), _ptr(s_col), M, _stream(stream))
    _check(st, "mx_gemm_mxout_ex")
    return q_row, s_row, q_col, s_col


def mx_gemm_grouped(qa, sa, ea, qb, sb, eb, group_offsets, M, N, K, out_dtype=OUT_BF16, out=None, stream=None):
    """MXFP8 grouped GEMM (include/mx.h, mx_gemm_grouped): rows off[g] .. off[g+1] of A times the
    g-th [N][K] block of B.  group_offsets: int64 CUDA tensor [G + 1]."""
    if group_offsets.dtype != torch.int64:
        raise ValueError("group_offsets must be int64")
    out, ldc = _out(M, N, out_dtype, out, qa.device)
    st = load().mx_gemm_grouped(_ptr(qa), _ptr(sa), ea, _ptr(qb), _ptr(sb), eb, _ptr(group_offsets),
                                group_offsets.numel() - 1, M, N, K, out.data_ptr(), out_dtype, ldc, _stream(stream))
    _check(st, "mx_gemm_grouped")
    return out


def nvfp4_gemm(qa, sa, ga, qb, sb, gb, M, N, K, out_dtype=OUT_F32, out=None, stream=None):
    """C = gA gB sum_b sA sB sum_i qA qB (NVFP4, include/mx.h nvfp4_gemm)."""
    out, ldc = _out(M, N, out_dtype, out, qa.device)
    st = load().nvfp4_gemm(_ptr(qa), _ptr(sa), _ptr(ga), _ptr(qb), _ptr(sb), _ptr(gb), M, N, K, out.data_ptr(),
                           out_dtype, ldc, _stream(stream))
    _check(st, "nvfp4_gemm")
    return out


def fp8_blockwise_gemm_grouped(qa, sa, qb, sb, group_offsets, M, N, K, out_dtype=OUT_BF16, out=None, stream=None):
    """DeepSeek FP8 grouped GEMM (include/mx.h, fp8_blockwise_gemm_grouped): rows off[g] .. off[g+1] of
    A times the g-th [N][K] block of B, FP32 promotion every 128 of K.  sa float [K/128][M] (1x128
    tiles), sb float [G*N/128][K/128] (128x128 blocks of the stacked weights)."""
    if group_offsets.dtype != torch.int64:
        raise ValueError("group_offsets must be int64")
    out, ldc = _out(M, N, out_dtype, out, qa.device)
    st = load().fp8_blockwise_gemm_grouped(_ptr(qa), _ptr(sa), _ptr(qb), _ptr(sb), _ptr(group_offsets),
                                           group_offsets.numel() - 1, M, N, K, out.data_ptr(), out_dtype, ldc,
                                           _stream(stream))
    _check(st, "fp8_blockwise_gemm_grouped")
    return out


def fp8_blockwise_gemm(qa, sa, qb, sb, M, N, K, out_dtype=OUT_BF16, out=None, stream=None):
    """DeepSeek FP8 GEMM with FP32 promotion every 128 of K (include/mx.h)."""
    out, ldc = _out(M, N, out_dtype, out, qa.device)
    st = load().fp8_blockwise_gemm(_ptr(qa), _ptr(sa), _ptr(qb), _ptr(sb), M, N, K, out.data_ptr(), out_dtype, ldc,
                                   _stream(stream))
    _check(st, "fp8_blockwise_gemm")
    return out


# ------------------------------------------------------------------ 8-bit key/value cache
# (Calls of a few microseconds: each tensor is looked at once, on the way to its address.)
_HALF = {torch.bfloat16: HALF_BF16, torch.float16: HALF_F16}
_int32, _int64, _float32, _uint8 = torch.int32, torch.int64, torch.float32, torch.uint8


def _at(t, dtype, name):
    """Address of a contiguous CUDA tensor of that type."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.data_ptr()


def _rows_of_heads(x, name):
    """(shape, address, type, token stride, head stride) of x[tokens][heads][head_dim], strided but for
    the last axis.  (An axis of one has no stride to speak of: torch may give it any.)"""
    half = _HALF.get(x.dtype)
    if half is None or x.dim() != 3:
        raise ValueError(f"{name} must be a 3-D bf16 or fp16 tensor")
    st, sh, sd = x.stride()
    if not x.is_cuda or sd != 1:
        raise ValueError(f"{name} must be a CUDA tensor whose last axis is contiguous")
    shape = x.shape
    return shape, x.data_ptr(), half, st if shape[0] > 1 else 0, sh if shape[1] > 1 else 0


def _cache_shape(k_codes, v_codes, k_scale, v_scale):
    shape = k_codes.shape
    if len(shape) != 4 or v_codes.shape != shape:
        raise ValueError("codes must be uint8 [num_blocks][kv_heads][block_tokens][head_dim]")
    if k_scale.shape != shape[:2] or v_scale.shape != k_scale.shape:
        raise ValueError("scales must be float32 [num_blocks][kv_heads]")
    return shape


def kv_block_tables(block_tables: torch.Tensor, len_before: torch.Tensor, len_after: torch.Tensor,
                    free_list: torch.Tensor, free_count: torch.Tensor, num_tokens: int, block_tokens: int,
                    q_start=None, slot_map=None, positions=None, info=None, stream=None):
    """Cache blocks for requests whose lengths go from len_before to len_after, and the new tokens'
    places (include/mx.h, kv_block_tables).  block_tables int32 [requests][max_blocks] and free_list
    int32 [capacity] are updated in place.  Returns (q_start int32 [requests + 1], slot_map int64
    [num_tokens], positions int32 [num_tokens], info int32 {free blocks left, blocks missing})."""
    requests, max_blocks = block_tables.shape if block_tables.dim() == 2 else (0, 0)
    if not requests or len_before.numel() != requests or len_after.numel() != requests or free_count.numel() < 1:
        raise ValueError("block_tables is [requests][max_blocks], the lengths are [requests], free_count [1]")
    at = (_at(block_tables, _int32, "block_tables"), _at(len_before, _int32, "len_before"),
          _at(len_after, _int32, "len_after"), _at(free_list, _int32, "free_list"), _at(free_count, _int32, "free_count"))
    dev = block_tables.device
    if q_start is None:
        q_start = torch.empty(requests + 1, dtype=_int32, device=dev)
    if slot_map is None:
        slot_map = torch.empty(num_tokens, dtype=_int64, device=dev)
    if positions is None:
        positions = torch.empty(num_tokens, dtype=_int32, device=dev)
    if info is None:
        info = torch.empty(2, dtype=_int32, device=dev)
    if (q_start.numel() <= requests or slot_map.numel() < num_tokens or positions.numel() < num_tokens
            or info.numel() < 2):
        raise ValueError("q_start has requests + 1 places, slot_map and positions num_tokens, info two")
    st = load().kv_block_tables(at[0], requests, max_blocks, at[1], at[2], at[3], free_list.numel(), at[4], block_tokens,
                                num_tokens, _at(q_start, _int32, "q_start"), _at(slot_map, _int64, "slot_map"),
                                _at(positions, _int32, "positions"), _at(info, _int32, "info"), _stream(stream))
    if st:
        _check(st, "kv_block_tables")
    return q_start, slot_map, positions, info


def kv_cache_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, k_codes: torch.Tensor,
                    v_codes: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, elem: int = E4M3, stream=None):
    """Quantize keys and values k, v [tokens][kv_heads][head_dim] (bf16 or fp16, slices will do) into
    the cache at slot_map (int64), in place (include/mx.h, kv_cache_append)."""
    shape, k_at, half, k_st, k_sh = _rows_of_heads(k, "k")
    v_shape, v_at, v_half, v_st, v_sh = _rows_of_heads(v, "v")
    blocks, kv_heads, block_tokens, head_dim = _cache_shape(k_codes, v_codes, k_scale, v_scale)
    tokens = shape[0]
    if v_half != half or v_shape != shape or shape[1] != kv_heads or shape[2] != head_dim:
        raise ValueError("k and v must be alike, [tokens][kv_heads][head_dim] of the cache")
    if slot_map.numel() != tokens:
        raise ValueError("slot_map must have a place for each token")
    st = load().kv_cache_append(k_at, v_at, half, tokens, k_st, k_sh, v_st, v_sh, _at(slot_map, _int64, "slot_map"),
                                _at(k_codes, _uint8, "k_codes"), _at(v_codes, _uint8, "v_codes"),
                                _at(k_scale, _float32, "k_scale"), _at(v_scale, _float32, "v_scale"), elem, blocks,
                                kv_heads, block_tokens, head_dim, _stream(stream))
    if st:
        _check(st, "kv_cache_append")


@functools.lru_cache(maxsize=256)
def kv_attention_workspace_bytes(num_tokens: int, requests: int, max_q_len: int, heads: int, kv_heads: int,
                                 head_dim: int) -> int:
    return int(load().kv_attention_workspace_bytes(num_tokens, requests, max_q_len, heads, kv_heads, head_dim))


_LEGACY, _PER_THREAD = 1, 2  # handles of CUDA's default streams; 0 is the first of them
_workspaces = {}        # (device, stream) -> the buffer that calls on that stream share
_workspaces_old = []    # outgrown ones, kept: work in flight may use them (each is larger than the last, and sizes are few)
_MOST_REQUESTS = 16384


def _kv_workspace(need, dev, stream, given):
    """A workspace for a call that was given none, made and cleared on the stream that the call goes to: calls
    on one stream follow each other and share one; a capture gets its own, since its graph may be replayed
    beside the stream."""
    if given is not None and stream != _stream(None):
        if stream == _LEGACY:
            stream = 0
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)):
            return _kv_workspace(need, dev, stream, None)
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(need, dtype=_uint8, device=dev)
        ws[:4096].zero_()  # (all that has to be clear)
        return ws
    ws = _workspaces.get((dev.index, stream))
    if ws is None or ws.numel() < need:
        with _lock:  # (and looked at again: another thread may have made it)
            ws = _workspaces.get((dev.index, stream))
            if ws is None or ws.numel() < need:
                if ws is not None:
                    _workspaces_old.append(ws)
                ws = _workspaces[(dev.index, stream)] = torch.zeros(need, dtype=_uint8, device=dev)
    return ws


def kv_attention(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, block_tables: torch.Tensor, lengths: torch.Tensor, q_start: torch.Tensor,
                 max_q_len: int, elem: int = E4M3, softmax_scale=None, causal: bool = True, window: int = 0, out=None,
                 lse=None, workspace=None, stream=None):
    """Attention of q [tokens][heads][head_dim] over the 8-bit cache (include/mx.h, kv_attention).
    lengths int32 [requests]: cached tokens, the queries' own among them; q_start int32 [requests + 1];
    softmax_scale defaults to head_dim ** -0.5; a workspace is zero before its first use, and calls
    without one share one for each stream (on the per-thread default stream the caller gives one).
    Returns (out, like q but contiguous; lse float [tokens][heads])."""
    return _kv_attention("kv_attention", (), (causal,), q, k_codes, v_codes, k_scale, v_scale, block_tables, lengths, q_start,
                         max_q_len, elem, softmax_scale, window, out, lse, workspace, stream)


def kv_tree_attention(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                      v_scale: torch.Tensor, block_tables: torch.Tensor, lengths: torch.Tensor, q_start: torch.Tensor,
                      max_q_len: int, tree_mask: torch.Tensor, positions=None, elem: int = E4M3, softmax_scale=None,
                      window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """kv_attention of a tree's queries: of their request's newest tokens, the tree's nodes, they see those whose bits
    tree_mask int64 [tokens][words] has (include/mx.h, kv_tree_attention).  positions int32 [tokens] with a window;
    kv_draft_trees gives both.  All else as kv_attention."""
    tokens = q.shape[0]
    if tree_mask.dim() != 2 or tree_mask.shape[0] != tokens or (positions is not None and positions.numel() != tokens):
        raise ValueError("tree_mask must be [tokens][words], positions [tokens]")
    if window and positions is None:
        raise ValueError("a window needs positions")
    tree = (_at(tree_mask, _int64, "tree_mask"), tree_mask.shape[1],
            None if positions is None else _at(positions, _int32, "positions"))
    _one_device(q, k_codes, v_codes, k_scale, v_scale, block_tables, lengths, q_start, tree_mask, positions, out, lse, workspace)
    return _kv_attention("kv_tree_attention", tree, (), q, k_codes, v_codes, k_scale, v_scale, block_tables, lengths, q_start,
                         max_q_len, elem, softmax_scale, window, out, lse, workspace, stream)


def _kv_attention(entry, tree, causal, q, k_codes, v_codes, k_scale, v_scale, block_tables, lengths, q_start, max_q_len, elem,
                  softmax_scale, window, out, lse, workspace, stream):
    shape, q_at, half, q_st, q_sh = _rows_of_heads(q, "q")
    blocks, kv_heads, block_tokens, head_dim = _cache_shape(k_codes, v_codes, k_scale, v_scale)
    tokens, heads, d = shape
    requests = lengths.numel()
    table_rows, max_blocks = block_tables.shape if block_tables.dim() == 2 else (-1, 0)
    if d != head_dim or table_rows != requests or q_start.numel() != requests + 1:
        raise ValueError("q [tokens][heads][head_dim], block_tables [requests][max_blocks], lengths [requests], "
                         "q_start [requests + 1]")
    dev = q.device
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    elif out.shape != shape or _at(out, q.dtype, "out") is None:
        raise ValueError("out must be shaped like q")
    if lse is None:
        lse = torch.empty((tokens, heads), dtype=_float32, device=dev)
    elif lse.shape != shape[:2] or _at(lse, _float32, "lse") is None:
        raise ValueError("lse must be [tokens][heads]")
    at_stream = _stream(stream)
    if workspace is None:
        if at_stream == _PER_THREAD:  # (another stream in every thread under one handle: nothing can be kept for it)
            raise ValueError("a call on the per-thread default stream needs a workspace of the caller's")
        # (for the most requests, 0.1 MB more: a size follows from the kernel and head_dim alone)
        need = kv_attention_workspace_bytes(1, _MOST_REQUESTS, max_q_len, heads, kv_heads, head_dim)
        workspace = _kv_workspace(need, dev, at_stream, stream)
    else:
        need = kv_attention_workspace_bytes(tokens, requests, max_q_len, heads, kv_heads, head_dim)
        if workspace.numel() < need or _at(workspace, _uint8, "workspace") is None:
            raise ValueError(f"workspace must have {need} bytes")
    st = getattr(load(), entry)(q_at, half, tokens, heads, q_st, q_sh, _at(k_codes, _uint8, "k_codes"),
                             _at(v_codes, _uint8, "v_codes"), _at(k_scale, _float32, "k_scale"),
                             _at(v_scale, _float32, "v_scale"), elem, blocks, kv_heads, block_tokens, head_dim,
                             _at(block_tables, _int32, "block_tables"), max_blocks, _at(lengths, _int32, "lengths"),
                             _at(q_start, _int32, "q_start"), requests, max_q_len, *tree,
                             head_dim ** -0.5 if softmax_scale is None else softmax_scale, *causal, window,
                             out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), at_stream)
    if st:
        _check(st, entry)
    return out, lse


# ------------------------------------------------------------------ norm and rotation; drafted tokens
def _one_device(first, *others):
    """All on the current device, whose stream the call goes to: a kernel there cannot read another's memory."""
    if not first.is_cuda or first.get_device() != torch.cuda.current_device():
        raise ValueError("tensors must be CUDA tensors on the current device")
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")


def _qk_out(out, like, name):
    """(tensor, address, token stride, head stride) of an output shaped like a [tokens][heads][head_dim] tensor."""
    if out is None:  # (fresh outputs are not checked again)
        shape = like.shape
        out = torch.empty(shape, dtype=like.dtype, device=like.device)
        return out, out.data_ptr(), shape[1] * shape[2], shape[2]
    shape, at, _, st, sh = _rows_of_heads(out, name)
    if shape != like.shape or out.dtype is not like.dtype:
        raise ValueError(f"{name} must be shaped and typed like its input")
    return out, at, st, sh


def _qk_rest(q, q_weight, k_weight, cos_sin, positions, kv_heads):
    """(q_weight's address, k_weight's, whether they are FP32, table's address, its positions, rot_dim, positions' address)"""
    tokens, _, head_dim = q.shape
    wide = q_weight.dtype is _float32
    kind = _float32 if wide else q.dtype
    if q_weight.numel() != head_dim or (kv_heads and (k_weight is None or k_weight.numel() != head_dim)):
        raise ValueError("weights must have head_dim values")
    if positions is None:
        if cos_sin is not None:
            raise ValueError("a rotation needs positions")
    elif positions.numel() != tokens:
        raise ValueError("positions must have a place for each token")
    if cos_sin is not None and cos_sin.dim() != 2:
        raise ValueError("cos_sin must be float32 [positions][rot_dim]")
    return (_at(q_weight, kind, "q_weight"), _at(k_weight, kind, "k_weight") if kv_heads else None, wide,
            None if cos_sin is None else _at(cos_sin, _float32, "cos_sin"), 0 if cos_sin is None else cos_sin.shape[0],
            0 if cos_sin is None else cos_sin.shape[1], None if positions is None else _at(positions, _int32, "positions"))


def qk_norm_rope(q: torch.Tensor, k, q_weight: torch.Tensor, k_weight, cos_sin, positions, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of each head of q [tokens][heads][head_dim] and k [tokens][kv_heads][head_dim] (or None) and rotation
    to positions (int32; -1 leaves a token out) by cos_sin float32 [positions][rot_dim] (or None)
    (include/mx.h, qk_norm_rope).  Slices will do; outputs may be q and k themselves.  Returns (q_out, k_out)."""
    shape, q_at, half, q_st, q_sh = _rows_of_heads(q, "q")
    k_at, k_st, k_sh, kv_heads = None, 0, 0, 0
    if k is not None:
        k_shape, k_at, k_half, k_st, k_sh = _rows_of_heads(k, "k")
        if k_half != half or k_shape[0] != shape[0] or k_shape[2] != shape[2]:
            raise ValueError("q and k must be alike but for their heads")
        kv_heads = k_shape[1]
    qw, kw, wide, table, places, rot, pos = _qk_rest(q, q_weight, k_weight, cos_sin, positions, kv_heads)
    q_out, qo_at, qo_st, qo_sh = _qk_out(q_out, q, "q_out")
    ko_at, ko_st, ko_sh = None, 0, 0
    if k is not None:
        k_out, ko_at, ko_st, ko_sh = _qk_out(k_out, k, "k_out")
    _one_device(q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out)
    st = load().qk_norm_rope(q_at, k_at, half, shape[0], shape[1], kv_heads, shape[2], q_st, q_sh, k_st, k_sh, qw, kw, wide,
                             table, places, rot, pos, eps, interleaved, qo_at, ko_at, qo_st, qo_sh, ko_st, ko_sh,
                             _stream(stream))
    if st:
        _check(st, "qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out, q: torch.Tensor, k, q_weight: torch.Tensor, k_weight, cos_sin,
                          positions, eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, dq_weight=None,
                          dk_weight=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope(q, k, ...) from those of its results (include/mx.h, qk_norm_rope_backward).
    Returns (dq, dk, dq_weight float32 [head_dim], dk_weight)."""
    shape, q_at, half, q_st, q_sh = _rows_of_heads(q, "q")
    g_shape, g_at, g_half, g_st, g_sh = _rows_of_heads(dq_out, "dq_out")
    if g_shape != shape or g_half != half or (k is None) != (dk_out is None):
        raise ValueError("gradients must be shaped and typed like q and k")
    k_at, k_st, k_sh, kv_heads, gk_at, gk_st, gk_sh = None, 0, 0, 0, None, 0, 0
    if k is not None:
        k_shape, k_at, k_half, k_st, k_sh = _rows_of_heads(k, "k")
        gk_shape, gk_at, gk_half, gk_st, gk_sh = _rows_of_heads(dk_out, "dk_out")
        if k_half != half or k_shape[0] != shape[0] or k_shape[2] != shape[2]:
            raise ValueError("q and k must be alike but for their heads")
        if gk_shape != k_shape or gk_half != half:
            raise ValueError("gradients must be shaped and typed like q and k")
        kv_heads = k_shape[1]
    qw, kw, wide, table, places, rot, pos = _qk_rest(q, q_weight, k_weight, cos_sin, positions, kv_heads)
    dq, dq_at, dq_st, dq_sh = _qk_out(dq, q, "dq")
    dk_at, dk_st, dk_sh = None, 0, 0
    if k is not None:
        dk, dk_at, dk_st, dk_sh = _qk_out(dk, k, "dk")
    dev, head_dim = q.device, shape[2]
    if dq_weight is None:
        dq_weight = torch.empty(head_dim, dtype=_float32, device=dev)
    if dk_weight is None:
        dk_weight = torch.empty(head_dim, dtype=_float32, device=dev)
    if dq_weight.numel() != head_dim or dk_weight.numel() != head_dim:
        raise ValueError("the weights' gradients must have head_dim values")
    _one_device(q, k, dq_out, dk_out, q_weight, k_weight, cos_sin, positions, dq, dk, dq_weight, dk_weight, workspace)
    at_stream = _stream(stream)
    need = int(load().qk_norm_rope_workspace_bytes(head_dim))
    if workspace is None:
        workspace = _call_workspace(need, dev, at_stream)
    elif workspace.numel() < need:
        raise ValueError(f"workspace must have {need} bytes")
    st = load().qk_norm_rope_backward(g_at, gk_at, q_at, k_at, half, shape[0], shape[1], kv_heads, head_dim, g_st, g_sh, gk_st,
                                      gk_sh, q_st, q_sh, k_st, k_sh, qw, kw, wide, table, places, rot, pos, eps, interleaved,
                                      dq_at, dk_at, dq_st, dq_sh, dk_st, dk_sh, _at(dq_weight, _float32, "dq_weight"),
                                      _at(dk_weight, _float32, "dk_weight"), _at(workspace, _uint8, "workspace"), at_stream)
    if st:
        _check(st, "qk_norm_rope_backward")
    return dq, dk, dq_weight, dk_weight


def _call_workspace(need, dev, stream):
    """A workspace that need not be clear, for one call: torch's allocator has it back when the call's work on the
    stream is in order in front of the next owner's, so it is made as one of that stream's."""
    if stream == _stream(None):
        return torch.empty(need, dtype=_uint8, device=dev)
    if stream == _PER_THREAD:
        raise ValueError("a call on the per-thread default stream needs a workspace of the caller's")
    with torch.cuda.stream(torch.cuda.ExternalStream(0 if stream == _LEGACY else stream, device=dev)):
        return torch.empty(need, dtype=_uint8, device=dev)


def kv_draft_trees(parents: torch.Tensor, lengths: torch.Tensor, q_start: torch.Tensor, max_q_len: int, window: int = 0,
                   tree_mask=None, positions=None, stream=None):
    """Visibility and positions of trees of drafted tokens from their parents (int32 [tokens], numbers within a request;
    -1: none) (include/mx.h, kv_draft_trees).  Returns (tree_mask int64 [tokens][ceil(max_q_len / 64)], positions int32
    [tokens])."""
    tokens, requests, dev = parents.numel(), lengths.numel(), parents.device
    if q_start.numel() != requests + 1:
        raise ValueError("q_start must be [requests + 1]")
    if tree_mask is None:
        tree_mask = torch.empty((tokens, max(1, (max_q_len + 63) // 64)), dtype=_int64, device=dev)
    if positions is None:
        positions = torch.empty(tokens, dtype=_int32, device=dev)
    if tree_mask.dim() != 2 or tree_mask.shape[0] != tokens or positions.numel() != tokens:
        raise ValueError("tree_mask must be [tokens][words] and positions [tokens]")
    _one_device(parents, lengths, q_start, tree_mask, positions)
    st = load().kv_draft_trees(_at(parents, _int32, "parents"), tokens, _at(lengths, _int32, "lengths"),
                               _at(q_start, _int32, "q_start"), requests, max_q_len, window,
                               _at(tree_mask, _int64, "tree_mask"), tree_mask.shape[1], _at(positions, _int32, "positions"),
                               _stream(stream))
    if st:
        _check(st, "kv_draft_trees")
    return tree_mask, positions


def _probs(x, tokens, name):
    """(address, row stride, vocabulary) of probabilities [tokens][vocab], rows apart but contiguous."""
    if x.dtype is not _float32 or x.dim() != 2 or not x.is_cuda or x.shape[0] != tokens:
        raise ValueError(f"{name} must be a float32 CUDA tensor [tokens][vocab]")
    st, sv = x.stride()
    vocab = x.shape[1]
    if sv != 1 and vocab > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return x.data_ptr(), st if tokens > 1 else vocab, vocab


def kv_verify_drafts(target_probs: torch.Tensor, drafts: torch.Tensor, parents: torch.Tensor, q_start: torch.Tensor,
                     accept_random: torch.Tensor, sample_random: torch.Tensor, draft_probs=None, max_q_len=None, path=None,
                     tokens=None, counts=None, stream=None):
    """Which drafted tokens the target's probabilities [tokens][vocab] keep, by given random numbers, and the token
    behind them (include/mx.h, kv_verify_drafts).  drafts, parents int32 [tokens]; q_start int32 [requests + 1];
    accept_random float32 [tokens], sample_random float32 [requests]; draft_probs: what the drafts were drawn from, or
    None where they are certain.  Returns (path int32 [tokens], tokens int32 [tokens], counts int32 [requests])."""
    n, requests, dev = drafts.numel(), sample_random.numel(), drafts.device
    t_at, t_st, vocab = _probs(target_probs, n, "target_probs")
    d_at, d_st = None, 0
    if draft_probs is not None:
        d_at, d_st, d_vocab = _probs(draft_probs, n, "draft_probs")
        if d_vocab != vocab:
            raise ValueError("draft_probs must be shaped like target_probs")
    if parents.numel() != n or accept_random.numel() != n or q_start.numel() != requests + 1:
        raise ValueError("parents and accept_random are [tokens], q_start is [requests + 1]")
    if path is None:
        path = torch.empty(n, dtype=_int32, device=dev)
    if tokens is None:
        tokens = torch.empty(n, dtype=_int32, device=dev)
    if counts is None:
        counts = torch.empty(requests, dtype=_int32, device=dev)
    if path.numel() != n or tokens.numel() != n or counts.numel() != requests:
        raise ValueError("path and tokens are [tokens], counts is [requests]")
    _one_device(drafts, target_probs, draft_probs, parents, q_start, accept_random, sample_random, path, tokens, counts)
    st = load().kv_verify_drafts(t_at, t_st, d_at, d_st, vocab, _at(drafts, _int32, "drafts"), _at(parents, _int32, "parents"),
                                 n, _at(q_start, _int32, "q_start"), requests, min(n, 1024) if max_q_len is None else max_q_len,
                                 _at(accept_random, _float32, "accept_random"), _at(sample_random, _float32, "sample_random"),
                                 _at(path, _int32, "path"), _at(tokens, _int32, "tokens"), _at(counts, _int32, "counts"),
                                 _stream(stream))
    if st:
        _check(st, "kv_verify_drafts")
    return path, tokens, counts


def kv_cache_compact(path: torch.Tensor, counts: torch.Tensor, lengths: torch.Tensor, q_start: torch.Tensor,
                     block_tables: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                     v_scale: torch.Tensor, elem: int = E4M3, kept_lengths=None, stream=None):
    """Moves the accepted nodes' keys and values together in the cache, in place (include/mx.h, kv_cache_compact).
    path and counts as kv_verify_drafts gives them.  Returns kept_lengths int32 [requests]."""
    blocks, kv_heads, block_tokens, head_dim = _cache_shape(k_codes, v_codes, k_scale, v_scale)
    requests = lengths.numel()
    table_rows, max_blocks = block_tables.shape if block_tables.dim() == 2 else (-1, 0)
    if table_rows != requests or counts.numel() != requests or q_start.numel() != requests + 1:
        raise ValueError("block_tables is [requests][max_blocks], lengths and counts are [requests], q_start [requests + 1]")
    if kept_lengths is None:
        kept_lengths = torch.empty(requests, dtype=_int32, device=lengths.device)
    elif kept_lengths.numel() != requests:
        raise ValueError("kept_lengths must be [requests]")
    _one_device(path, counts, lengths, q_start, block_tables, k_codes, v_codes, k_scale, v_scale, kept_lengths)
    st = load().kv_cache_compact(_at(path, _int32, "path"), _at(counts, _int32, "counts"), path.numel(),
                                 _at(lengths, _int32, "lengths"), _at(q_start, _int32, "q_start"), requests,
                                 _at(block_tables, _int32, "block_tables"), max_blocks, _at(k_codes, _uint8, "k_codes"),
                                 _at(v_codes, _uint8, "v_codes"), _at(k_scale, _float32, "k_scale"),
                                 _at(v_scale, _float32, "v_scale"), elem, blocks, kv_heads, block_tokens, head_dim,
                                 _at(kept_lengths, _int32, "kept_lengths"), _stream(stream))
    if st:
        _check(st, "kv_cache_compact")
    return kept_lengths


def mx_check(stream=None) -> int:
    """Synchronize the stream and return the library's device status (MX_OK / MX_ERR_TIMEOUT / ...)."""
    status = int(load().mx_check(_stream(stream)))
    if status == MX_ERR_TIMEOUT:  # a kernel that gave up may have left its workspace as it was
        with _lock:
            _workspaces_old.extend(_workspaces.values())
            _workspaces.clear()
    return status


def num_sms() -> int:
    return int(load().mx_num_sms())
