"""MI355X (gfx950) FP8 E4M3 block-scaled GEMM: Python binding of libdg.so.

Argument marshalling only: every step runs in the HIP kernels of libdg.so
(declared in include/dg.h).  PyTorch provides device memory and the current
stream.  There is no fallback: if the library is missing or fails to load,
importing this package raises.

Entry points (same names as the C ABI):
    dg_quantize_fp8_block(q, scales, x, block_rows)
    dg_fp8_gemm_nt(c, a, b, sa, sb, a_block_rows, workspace=None)
    dg_fp8_grouped_gemm_contig(c, a, b, sa, sb, a_block_rows, m_indices, workspace=None)
    dg_fp8_grouped_gemm_masked(c, a, b, sa, sb, a_block_rows, masked_m, workspace=None)
    dg_quantize_mxfp4(x, q, sf, qt, sft), dg_dequantize_mxfp4(out, q, sf)
    dg_mxfp4_gemm_nt(c, a, b, sfa, sfb), dg_mxfp4_gemm_nt_bf16a(c, a, b, sfb)
    dg_moe_layer(y, x, w13, w2, s13, s2, ids, weights, logits)
    dg_moe_route(ids, weights, logits), dg_moe_plan(rows, pairs, m_indices, offsets, counts, ids),
    dg_moe_dispatch_fp8(a, sa, x, rows, pairs), dg_moe_combine(y, c, rows, weights),
    dg_swiglu_fp8(h, sh, gu), dg_transpose_fp8_blocks(qt, st, q, s), and the backward calls
    (and the UE8M0, fused-A, epilogue, layout and K-grouped entry points)
Conveniences mirroring the DeepGEMM page's Python API (pzsr.cn, s4.1):
    to_fp8(x, block_rows=128) -> (q, scales)
    fp8_gemm_nt(c, a, b, sa, sb, a_block_rows=128)
"""
from __future__ import annotations

import collections
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libdg.so")

DG_OK = 0
ABI_VERSION = 3
# arrival-counter region at the start of every split-K workspace (dg.h)
WORKSPACE_COUNTER_BYTES = 32768


class DGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (where, status_string(status), status))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libdg.so not built (%s); run `python fp8_block_scaled_dg_amd/build.py`"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.dg_abi_version.restype = i32
    lib.dg_abi_version.argtypes = []
    lib.dg_status_string.restype = ctypes.c_char_p
    lib.dg_status_string.argtypes = [i32]
    lib.dg_get_mk_alignment_for_contiguous_layout.restype = i32
    lib.dg_get_mk_alignment_for_contiguous_layout.argtypes = []
    lib.dg_quantize_fp8_block.restype = i32
    lib.dg_quantize_fp8_block.argtypes = [vp, vp, vp, i64, i64, i32, vp]
    lib.dg_fp8_gemm_nt_workspace_bytes.restype = ctypes.c_size_t
    lib.dg_fp8_gemm_nt_workspace_bytes.argtypes = [i64, i64, i64]
    lib.dg_fp8_gemm_nt.restype = i32
    lib.dg_fp8_gemm_nt.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.dg_quantize_fp8_block_ue8m0.restype = i32
    lib.dg_quantize_fp8_block_ue8m0.argtypes = [vp, vp, vp, i64, i64, i32, vp]
    lib.dg_fp8_gemm_nt_ue8m0.restype = i32
    lib.dg_fp8_gemm_nt_ue8m0.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp,
                                         ctypes.c_size_t, vp]
    lib.dg_fp8_gemm_nt_epilogue.restype = i32
    lib.dg_fp8_gemm_nt_epilogue.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, i32, vp, vp,
                                            ctypes.c_size_t, vp]
    lib.dg_transpose_fp8.restype = i32
    lib.dg_transpose_fp8.argtypes = [vp, vp, i64, i64, vp]
    lib.dg_fp8_gemm_workspace_bytes.restype = ctypes.c_size_t
    lib.dg_fp8_gemm_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.dg_fp8_gemm.restype = i32
    lib.dg_fp8_gemm.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, i32, vp, ctypes.c_size_t,
                                vp]
    lib.dg_fp8_grouped_gemm_k.restype = i32
    lib.dg_fp8_grouped_gemm_k.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64, i64, vp]
    lib.dg_fp8_gemm_nt_fused_a.restype = i32
    lib.dg_fp8_gemm_nt_fused_a.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t,
                                           vp]
    lib.dg_fp8_gemm_nt_fused_a_bf16.restype = i32
    lib.dg_fp8_gemm_nt_fused_a_bf16.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp,
                                                ctypes.c_size_t, vp]
    lib.dg_fp8_grouped_gemm_contig.restype = i32
    lib.dg_fp8_grouped_gemm_contig.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64, i64, vp]
    lib.dg_fp8_grouped_gemm_masked_workspace_bytes.restype = ctypes.c_size_t
    lib.dg_fp8_grouped_gemm_masked_workspace_bytes.argtypes = [i32, i64, i64, i64]
    lib.dg_fp8_grouped_gemm_contig_epilogue.restype = i32
    lib.dg_fp8_grouped_gemm_contig_epilogue.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64,
                                                        i64, i32, vp, vp]
    lib.dg_fp8_grouped_gemm_masked_epilogue.restype = i32
    lib.dg_fp8_grouped_gemm_masked_epilogue.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64,
                                                        i64, i32, vp, vp, ctypes.c_size_t, vp]
    lib.dg_fp8_grouped_gemm_contig_workspace_bytes.restype = ctypes.c_size_t
    lib.dg_fp8_grouped_gemm_contig_workspace_bytes.argtypes = [i64, i64, i64]
    lib.dg_fp8_grouped_gemm_contig_balanced.restype = i32
    lib.dg_fp8_grouped_gemm_contig_balanced.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64,
                                                        i64, i32, vp, vp, ctypes.c_size_t, vp]
    lib.dg_fp8_grouped_gemm_contig_ue8m0.restype = i32
    lib.dg_fp8_grouped_gemm_contig_ue8m0.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64,
                                                     i64, vp]
    lib.dg_fp8_grouped_gemm_masked_ue8m0.restype = i32
    lib.dg_fp8_grouped_gemm_masked_ue8m0.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64,
                                                     i64, vp, ctypes.c_size_t, vp]
    lib.dg_fp8_grouped_gemm_masked.restype = i32
    lib.dg_fp8_grouped_gemm_masked.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, i64, i64, vp,
                                               ctypes.c_size_t, vp]
    lib.dg_fp8_gemm_nt_noalloc.restype = i32
    lib.dg_fp8_gemm_nt_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    sz = ctypes.c_size_t
    lib.dg_quantize_mxfp4.restype = i32
    lib.dg_quantize_mxfp4.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    lib.dg_dequantize_mxfp4.restype = i32
    lib.dg_dequantize_mxfp4.argtypes = [vp, i32, vp, vp, i64, i64, vp]
    lib.dg_mxfp4_gemm_nt_workspace_bytes.restype = sz
    lib.dg_mxfp4_gemm_nt_workspace_bytes.argtypes = [i64, i64, i64]
    lib.dg_mxfp4_gemm_nt.restype = i32
    lib.dg_mxfp4_gemm_nt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.dg_mxfp4_gemm_nt_bf16a_workspace_bytes.restype = sz
    lib.dg_mxfp4_gemm_nt_bf16a_workspace_bytes.argtypes = [i64, i64, i64]
    lib.dg_mxfp4_gemm_nt_bf16a.restype = i32
    lib.dg_mxfp4_gemm_nt_bf16a.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.dg_moe_layer_workspace_bytes.restype = sz
    lib.dg_moe_layer_workspace_bytes.argtypes = [i32, i32, i32, i64, i64]
    lib.dg_moe_layer.restype = i32
    lib.dg_moe_layer.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, i64,
                                 i64, vp, sz, vp]
    f32 = ctypes.c_float
    lib.dg_moe_route.restype = i32
    lib.dg_moe_route.argtypes = [vp, vp, vp, i32, i64, vp, i32, i32, i32, i32, i32, f32, i64, i32,
                                 i32, vp]
    lib.dg_moe_route_backward.restype = i32
    lib.dg_moe_route_backward.argtypes = [vp, i64, vp, vp, vp, i32, i64, i32, i32, f32, i64, i32,
                                          i32, vp]
    lib.dg_moe_plan_rows.restype = i64
    lib.dg_moe_plan_rows.argtypes = [i64, i32, i32]
    lib.dg_moe_plan_workspace_bytes.restype = sz
    lib.dg_moe_plan_workspace_bytes.argtypes = [i64, i32, i32]
    lib.dg_moe_plan.restype = i32
    lib.dg_moe_plan.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i32, i64, vp, sz, vp]
    lib.dg_moe_dispatch_fp8.restype = i32
    lib.dg_moe_dispatch_fp8.argtypes = [vp, vp, vp, i32, i64, vp, vp, vp, i64, i32, i64, i64, vp, sz,
                                        vp]
    lib.dg_moe_dispatch_fp8_workspace_bytes.restype = sz
    lib.dg_moe_dispatch_fp8_workspace_bytes.argtypes = [i64, i32, i64, i32]
    lib.dg_moe_combine.restype = i32
    lib.dg_moe_combine.argtypes = [vp, vp, vp, vp, vp, i64, i32, i64, i64, vp]
    lib.dg_moe_combine_backward.restype = i32
    lib.dg_moe_combine_backward.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp, vp, i64, i32, i64,
                                            i64, vp, sz, vp]
    lib.dg_swiglu_fp8.restype = i32
    lib.dg_swiglu_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp]
    lib.dg_swiglu_fp8_backward.restype = i32
    lib.dg_swiglu_fp8_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, vp]
    lib.dg_transpose_fp8_blocks.restype = i32
    lib.dg_transpose_fp8_blocks.argtypes = [vp, vp, i32, vp, vp, vp, i64, i64, vp]
    if lib.dg_abi_version() != ABI_VERSION:
        raise ImportError("libdg ABI %d != binding ABI %d" % (lib.dg_abi_version(), ABI_VERSION))
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.dg_status_string(status).decode()


def get_mk_alignment_for_contiguous_layout() -> int:
    return lib.dg_get_mk_alignment_for_contiguous_layout()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The stream's handle; by default the current stream's of the current
    device (asked for by handle: a torch.cuda.Stream object costs 3 us)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream


def _check(rc: int, where: str):
    if rc != DG_OK:
        raise DGError(rc, where)


def _require(t, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _codes(t, name):
    if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn:
        _require(t, torch.float8_e4m3fn, name)
    else:
        _require(t, torch.uint8, name)
    return t


_BF16_TYPES = (torch.bfloat16, getattr(torch, "uint16", torch.int16))  # or int16: raw bits


def _bf16(t, name):
    if isinstance(t, torch.Tensor) and t.dtype in _BF16_TYPES:
        _require(t, t.dtype, name)
    else:
        _require(t, torch.int16, name)
    return t


def _workspace_bytes(workspace) -> int:
    if workspace is None:
        return 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return workspace.numel() * workspace.element_size()


def alloc_workspace(nbytes: int, device="cuda"):
    """A split-K workspace of at least nbytes (16 minimum), zero-filled: its
    counter region must be zero before first use; every call leaves it zero,
    so the tensor can be reused by later calls ordered after this one."""
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def cdiv(a: int, b: int) -> int:
    return (a + b - 1) // b


# ---------------------------------------------------------------------------
# C-ABI entry points
# ---------------------------------------------------------------------------

def dg_quantize_fp8_block(q, scales, x, block_rows: int = 128, stream=None) -> None:
    """x float32 [rows, cols] -> q (uint8/float8_e4m3fn [rows, cols]),
    scales float32 [ceil(cols/128), ceil(rows/block_rows)]."""
    _require(x, torch.float32, "x")
    q = _codes(q, "q")
    _require(scales, torch.float32, "scales")
    rows, cols = x.shape
    if q.shape != x.shape:
        raise ValueError("q must have the shape of x")
    if scales.numel() != cdiv(cols, 128) * cdiv(rows, block_rows):
        raise ValueError("scales must hold ceil(cols/128)*ceil(rows/block_rows) floats")
    _check(lib.dg_quantize_fp8_block(_ptr(q), _ptr(scales), _ptr(x), rows, cols, block_rows,
                                     _stream(stream)), "dg_quantize_fp8_block")


def dg_fp8_gemm_nt_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.dg_fp8_gemm_nt_workspace_bytes(M, N, K)


def dg_fp8_gemm_nt(c, a, b, sa, sb, a_block_rows: int = 128, workspace=None,
                   stream=None) -> None:
    """C[M,N] (bf16) = block-scaled A[M,K] . B[N,K]^T."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sa, torch.float32, "sa")
    _require(sb, torch.float32, "sb")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K or c.shape != (M, N):
        raise ValueError("shape mismatch: a %s, b %s, c %s" % (tuple(a.shape), tuple(b.shape),
                                                              tuple(c.shape)))
    if sa.numel() != cdiv(K, 128) * cdiv(M, a_block_rows):
        raise ValueError("sa must hold (K/128)*ceil(M/a_block_rows) floats")
    if sb.numel() != cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold (K/128)*ceil(N/128) floats")
    ws_bytes = _workspace_bytes(workspace)
    _check(lib.dg_fp8_gemm_nt(_ptr(c), _ptr(a), _ptr(b), _ptr(sa), _ptr(sb), a_block_rows,
                              M, N, K, _ptr(workspace), ws_bytes, _stream(stream)),
           "dg_fp8_gemm_nt")


# static split-K scratch of dg_fp8_gemm_nt_noalloc, per GPU (dg.h)
NOALLOC_SCRATCH_BYTES = 16 << 20


def dg_fp8_gemm_nt_noalloc(c, a, b, sa, sb, a_block_rows: int = 128, stream=None) -> None:
    """dg_fp8_gemm_nt without a workspace argument, for callers that cannot
    allocate: the split-K scratch is the library's static per-GPU array
    (calls that overlap on one GPU race on it)."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sa, torch.float32, "sa")
    _require(sb, torch.float32, "sb")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K or c.shape != (M, N):
        raise ValueError("shape mismatch: a %s, b %s, c %s" % (tuple(a.shape), tuple(b.shape),
                                                              tuple(c.shape)))
    if sa.numel() != cdiv(K, 128) * cdiv(M, a_block_rows):
        raise ValueError("sa must hold (K/128)*ceil(M/a_block_rows) floats")
    if sb.numel() != cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold (K/128)*ceil(N/128) floats")
    _check(lib.dg_fp8_gemm_nt_noalloc(_ptr(c), _ptr(a), _ptr(b), _ptr(sa), _ptr(sb), a_block_rows,
                                      M, N, K, _stream(stream)), "dg_fp8_gemm_nt_noalloc")


def dg_quantize_fp8_block_ue8m0(q, sf, x, block_rows: int = 128, stream=None) -> None:
    """x float32 [rows, cols] -> q (uint8/float8_e4m3fn [rows, cols]),
    sf int32 [ceil(cols/512), ceil(rows/block_rows)] (UE8M0 exponents, four K
    blocks per word)."""
    _require(x, torch.float32, "x")
    q = _codes(q, "q")
    _require(sf, torch.int32, "sf")
    rows, cols = x.shape
    if q.shape != x.shape:
        raise ValueError("q must have the shape of x")
    if sf.numel() != cdiv(cdiv(cols, 128), 4) * cdiv(rows, block_rows):
        raise ValueError("sf must hold ceil(cols/512)*ceil(rows/block_rows) int32")
    _check(lib.dg_quantize_fp8_block_ue8m0(_ptr(q), _ptr(sf), _ptr(x), rows, cols, block_rows,
                                           _stream(stream)), "dg_quantize_fp8_block_ue8m0")


def dg_fp8_gemm_nt_ue8m0(c, a, b, sfa, sfb, a_block_rows: int = 128, workspace=None,
                         stream=None) -> None:
    """C[M,N] (bf16) = A[M,K] . B[N,K]^T with packed UE8M0 block scales."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sfa, torch.int32, "sfa")
    _require(sfb, torch.int32, "sfb")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K or c.shape != (M, N):
        raise ValueError("shape mismatch: a %s, b %s, c %s" % (tuple(a.shape), tuple(b.shape),
                                                              tuple(c.shape)))
    if sfa.numel() != cdiv(cdiv(K, 128), 4) * cdiv(M, a_block_rows):
        raise ValueError("sfa must hold ceil(K/512)*ceil(M/a_block_rows) int32")
    if sfb.numel() != cdiv(cdiv(K, 128), 4) * cdiv(N, 128):
        raise ValueError("sfb must hold ceil(K/512)*ceil(N/128) int32")
    _check(lib.dg_fp8_gemm_nt_ue8m0(_ptr(c), _ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb), a_block_rows,
                                    M, N, K, _ptr(workspace), _workspace_bytes(workspace),
                                    _stream(stream)), "dg_fp8_gemm_nt_ue8m0")


FUSED_A_MAX_M = 64


def dg_fp8_gemm_nt_fused_a(c, a, b, sb, workspace=None, stream=None) -> None:
    """C[M,N] (bf16) = A[M,K] (float32 or bfloat16, quantised with 1x128
    blocks inside the GEMM) . B[N,K]^T (E4M3, 128x128 scales sb);
    M <= FUSED_A_MAX_M."""
    c = _bf16(c, "c")
    if not isinstance(a, torch.Tensor) or a.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("a must be a float32 or bfloat16 tensor")
    bf16 = a.dtype == torch.bfloat16
    _require(a, a.dtype, "a")
    b = _codes(b, "b")
    _require(sb, torch.float32, "sb")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K or c.shape != (M, N):
        raise ValueError("shape mismatch: a %s, b %s, c %s" % (tuple(a.shape), tuple(b.shape),
                                                              tuple(c.shape)))
    if sb.numel() != cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold (K/128)*ceil(N/128) floats")
    ws_bytes = _workspace_bytes(workspace)
    fn = lib.dg_fp8_gemm_nt_fused_a_bf16 if bf16 else lib.dg_fp8_gemm_nt_fused_a
    _check(fn(_ptr(c), _ptr(a), _ptr(b), _ptr(sb), M, N, K, _ptr(workspace), ws_bytes,
              _stream(stream)), "dg_fp8_gemm_nt_fused_a" + ("_bf16" if bf16 else ""))


EPILOGUES = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}


def dg_fp8_gemm_nt_epilogue(c, a, b, sa, sb, a_block_rows: int = 128, act: str = "none",
                            residual=None, workspace=None, stream=None) -> None:
    """C = epilogue(A . B^T): act in EPILOGUES (swiglu: B rows interleave gate
    and up, C has N/2 columns), plus an optional BF16 residual [M, Nout]
    (may be c itself)."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sa, torch.float32, "sa")
    _require(sb, torch.float32, "sb")
    M, K = a.shape
    N = b.shape[0]
    code = EPILOGUES[act]
    n_out = N // 2 if code == EPILOGUES["swiglu"] else N
    if b.shape[1] != K or c.shape != (M, n_out):
        raise ValueError("shape mismatch: a %s, b %s, c %s (act %s)"
                         % (tuple(a.shape), tuple(b.shape), tuple(c.shape), act))
    if sa.numel() != cdiv(K, 128) * cdiv(M, a_block_rows):
        raise ValueError("sa must hold (K/128)*ceil(M/a_block_rows) floats")
    if sb.numel() != cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold (K/128)*ceil(N/128) floats")
    if residual is not None:
        residual = _bf16(residual, "residual")
        if residual.shape != (M, n_out):
            raise ValueError("residual must be [M, Nout]")
    _check(lib.dg_fp8_gemm_nt_epilogue(_ptr(c), _ptr(a), _ptr(b), _ptr(sa), _ptr(sb), a_block_rows,
                                       M, N, K, code, _ptr(residual), _ptr(workspace),
                                       _workspace_bytes(workspace), _stream(stream)),
           "dg_fp8_gemm_nt_epilogue")


LAYOUTS = {"nt": 0, "tn": 1, "nn": 2, "tt": 3}


def dg_transpose_fp8(out, inp, stream=None) -> None:
    """out [cols, rows] = inp [rows, cols]^T (bytes; rows, cols multiples of 16)."""
    out = _codes(out, "out")
    inp = _codes(inp, "inp")
    rows, cols = inp.shape
    if out.shape != (cols, rows):
        raise ValueError("out must be [cols, rows]")
    _check(lib.dg_transpose_fp8(_ptr(out), _ptr(inp), rows, cols, _stream(stream)),
           "dg_transpose_fp8")


def dg_fp8_gemm_workspace_bytes(M: int, N: int, K: int, layout: str = "nt") -> int:
    return lib.dg_fp8_gemm_workspace_bytes(M, N, K, LAYOUTS[layout])


def dg_fp8_gemm(c, a, b, sa, sb, a_block_rows: int = 128, layout: str = "nt", workspace=None,
                stream=None) -> None:
    """C[M,N] = A . B^T with operands stored per ``layout`` (first letter A:
    n = [M,K], t = [K,M]; second letter B: t = [N,K], n = [K,N])."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sa, torch.float32, "sa")
    _require(sb, torch.float32, "sb")
    M, N = c.shape
    a_t = layout in ("tn", "tt")
    b_n = layout in ("tn", "nn")
    K = a.shape[0] if a_t else a.shape[1]
    if a.shape != ((K, M) if a_t else (M, K)) or b.shape != ((K, N) if b_n else (N, K)):
        raise ValueError("shape mismatch for layout %s: a %s, b %s, c %s"
                         % (layout, tuple(a.shape), tuple(b.shape), tuple(c.shape)))
    if sa.numel() != cdiv(K, 128) * cdiv(M, a_block_rows):
        raise ValueError("sa must hold (K/128)*ceil(M/a_block_rows) floats")
    if sb.numel() != cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold (K/128)*ceil(N/128) floats")
    _check(lib.dg_fp8_gemm(_ptr(c), _ptr(a), _ptr(b), _ptr(sa), _ptr(sb), a_block_rows, M, N, K,
                           LAYOUTS[layout], _ptr(workspace), _workspace_bytes(workspace),
                           _stream(stream)), "dg_fp8_gemm")


def dg_fp8_grouped_gemm_k(c, a, b, sa, sb, a_block_rows: int, k_offsets, stream=None) -> None:
    """K-grouped: c [G, M, N] (bf16), a [M, K], b [N, K], k_offsets int64
    device [G + 1] (multiples of 128): c[g] = A[:, k0:k1] . B[:, k0:k1]^T."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sa, torch.float32, "sa")
    _require(sb, torch.float32, "sb")
    _require(k_offsets, torch.int64, "k_offsets")
    M, K = a.shape
    N = b.shape[0]
    G = k_offsets.numel() - 1
    if b.shape[1] != K or c.shape != (G, M, N):
        raise ValueError("shape mismatch")
    if sa.numel() != cdiv(K, 128) * cdiv(M, a_block_rows):
        raise ValueError("sa must hold (K/128)*ceil(M/a_block_rows) floats")
    if sb.numel() != cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold (K/128)*ceil(N/128) floats")
    _check(lib.dg_fp8_grouped_gemm_k(_ptr(c), _ptr(a), _ptr(b), _ptr(sa), _ptr(sb), a_block_rows,
                                     _ptr(k_offsets), G, M, N, K, _stream(stream)),
           "dg_fp8_grouped_gemm_k")


def dg_fp8_grouped_gemm_contig_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.dg_fp8_grouped_gemm_contig_workspace_bytes(M, N, K)


def dg_fp8_grouped_gemm_contig(c, a, b, sa, sb, a_block_rows: int, m_indices, act: str = "none",
                               residual=None, workspace=None, stream=None) -> None:
    """Grouped M-contiguous: a [M,K], b [G,N,K], sb [G,K/128,ceil(N/128)],
    m_indices int32 [M] (-1 = padding row -> zero row).  act / residual: the
    fused epilogue (swiglu: each expert's B rows interleave gate and up, c has
    N/2 columns); padding rows stay zero.  workspace (zero-filled device
    bytes, dg_fp8_grouped_gemm_contig_workspace_bytes(M, N, K) of them; see
    alloc_workspace): share the work evenly over the compute units
    (dg_fp8_grouped_gemm_contig_balanced)."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sa, torch.float32, "sa")
    _require(sb, torch.float32, "sb")
    _require(m_indices, torch.int32, "m_indices")
    M, K = a.shape
    G, N, Kb = b.shape
    code = EPILOGUES[act]
    n_out = N // 2 if code == EPILOGUES["swiglu"] else N
    if Kb != K or c.shape != (M, n_out) or m_indices.shape != (M,):
        raise ValueError("inconsistent grouped GEMM shapes")
    if sa.numel() != cdiv(K, 128) * cdiv(M, a_block_rows):
        raise ValueError("sa must hold (K/128)*ceil(M/a_block_rows) floats")
    if sb.numel() != G * cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold G*(K/128)*ceil(N/128) floats")
    if residual is not None:
        residual = _bf16(residual, "residual")
        if residual.shape != (M, n_out):
            raise ValueError("residual must be [M, Nout]")
    if workspace is not None:
        rc = lib.dg_fp8_grouped_gemm_contig_balanced(_ptr(c), _ptr(a), _ptr(b), _ptr(sa),
                                                     _ptr(sb), a_block_rows, _ptr(m_indices), G,
                                                     M, N, K, code, _ptr(residual),
                                                     _ptr(workspace), _workspace_bytes(workspace),
                                                     _stream(stream))
    elif code == 0 and residual is None:
        rc = lib.dg_fp8_grouped_gemm_contig(_ptr(c), _ptr(a), _ptr(b), _ptr(sa), _ptr(sb),
                                            a_block_rows, _ptr(m_indices), G, M, N, K,
                                            _stream(stream))
    else:
        rc = lib.dg_fp8_grouped_gemm_contig_epilogue(_ptr(c), _ptr(a), _ptr(b), _ptr(sa),
                                                     _ptr(sb), a_block_rows, _ptr(m_indices), G,
                                                     M, N, K, code, _ptr(residual),
                                                     _stream(stream))
    _check(rc, "dg_fp8_grouped_gemm_contig")


def dg_fp8_grouped_gemm_contig_ue8m0(c, a, b, sfa, sfb, a_block_rows: int, m_indices,
                                     stream=None) -> None:
    """Grouped M-contiguous with packed UE8M0 scales: sfa int32
    [ceil(K/512), ceil(M/br)], sfb int32 [G, ceil(K/512), ceil(N/128)]."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sfa, torch.int32, "sfa")
    _require(sfb, torch.int32, "sfb")
    _require(m_indices, torch.int32, "m_indices")
    M, K = a.shape
    G, N, Kb = b.shape
    if Kb != K or c.shape != (M, N) or m_indices.shape != (M,):
        raise ValueError("inconsistent grouped GEMM shapes")
    if sfa.numel() != cdiv(cdiv(K, 128), 4) * cdiv(M, a_block_rows):
        raise ValueError("sfa must hold ceil(K/512)*ceil(M/a_block_rows) int32")
    if sfb.numel() != G * cdiv(cdiv(K, 128), 4) * cdiv(N, 128):
        raise ValueError("sfb must hold G*ceil(K/512)*ceil(N/128) int32")
    _check(lib.dg_fp8_grouped_gemm_contig_ue8m0(_ptr(c), _ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb),
                                                a_block_rows, _ptr(m_indices), G, M, N, K,
                                                _stream(stream)), "dg_fp8_grouped_gemm_contig_ue8m0")


def dg_fp8_grouped_gemm_masked_ue8m0(c, a, b, sfa, sfb, a_block_rows: int, masked_m,
                                     workspace=None, stream=None) -> None:
    """Masked grouped with packed UE8M0 scales: sfa int32
    [G, ceil(K/512), ceil(max_m/br)], sfb int32 [G, ceil(K/512), ceil(N/128)]."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sfa, torch.int32, "sfa")
    _require(sfb, torch.int32, "sfb")
    _require(masked_m, torch.int32, "masked_m")
    G, max_m, K = a.shape
    Gb, N, Kb = b.shape
    if Gb != G or Kb != K or c.shape != (G, max_m, N) or masked_m.shape != (G,):
        raise ValueError("inconsistent masked grouped GEMM shapes")
    if sfa.numel() != G * cdiv(cdiv(K, 128), 4) * cdiv(max_m, a_block_rows):
        raise ValueError("sfa must hold G*ceil(K/512)*ceil(max_m/a_block_rows) int32")
    if sfb.numel() != G * cdiv(cdiv(K, 128), 4) * cdiv(N, 128):
        raise ValueError("sfb must hold G*ceil(K/512)*ceil(N/128) int32")
    _check(lib.dg_fp8_grouped_gemm_masked_ue8m0(_ptr(c), _ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb),
                                                a_block_rows, _ptr(masked_m), G, max_m, N, K,
                                                _ptr(workspace), _workspace_bytes(workspace),
                                                _stream(stream)), "dg_fp8_grouped_gemm_masked_ue8m0")


def dg_fp8_grouped_gemm_masked_workspace_bytes(num_groups: int, max_m: int, N: int,
                                              K: int) -> int:
    return lib.dg_fp8_grouped_gemm_masked_workspace_bytes(num_groups, max_m, N, K)


def dg_fp8_grouped_gemm_masked(c, a, b, sa, sb, a_block_rows: int, masked_m, workspace=None,
                               act: str = "none", residual=None, stream=None) -> None:
    """Masked grouped: a [G,max_m,K], b [G,N,K], sa [G,K/128,ceil(max_m/br)],
    sb [G,K/128,ceil(N/128)], masked_m int32 [G] (device), c [G,max_m,Nout]
    (Nout = N, or N/2 with act="swiglu"); rows past masked_m[g] of c[g] are
    not written.  act / residual [G,max_m,Nout]: the fused epilogue."""
    c = _bf16(c, "c")
    a = _codes(a, "a")
    b = _codes(b, "b")
    _require(sa, torch.float32, "sa")
    _require(sb, torch.float32, "sb")
    _require(masked_m, torch.int32, "masked_m")
    G, max_m, K = a.shape
    Gb, N, Kb = b.shape
    code = EPILOGUES[act]
    n_out = N // 2 if code == EPILOGUES["swiglu"] else N
    if Gb != G or Kb != K or c.shape != (G, max_m, n_out) or masked_m.shape != (G,):
        raise ValueError("inconsistent masked grouped GEMM shapes")
    if sa.numel() != G * cdiv(K, 128) * cdiv(max_m, a_block_rows):
        raise ValueError("sa must hold G*(K/128)*ceil(max_m/a_block_rows) floats")
    if sb.numel() != G * cdiv(K, 128) * cdiv(N, 128):
        raise ValueError("sb must hold G*(K/128)*ceil(N/128) floats")
    if residual is not None:
        residual = _bf16(residual, "residual")
        if residual.shape != (G, max_m, n_out):
            raise ValueError("residual must be [G, max_m, Nout]")
    if code == 0 and residual is None:
        rc = lib.dg_fp8_grouped_gemm_masked(_ptr(c), _ptr(a), _ptr(b), _ptr(sa), _ptr(sb),
                                            a_block_rows, _ptr(masked_m), G, max_m, N, K,
                                            _ptr(workspace), _workspace_bytes(workspace),
                                            _stream(stream))
    else:
        rc = lib.dg_fp8_grouped_gemm_masked_epilogue(_ptr(c), _ptr(a), _ptr(b), _ptr(sa),
                                                     _ptr(sb), a_block_rows, _ptr(masked_m), G,
                                                     max_m, N, K, code, _ptr(residual),
                                                     _ptr(workspace), _workspace_bytes(workspace),
                                                     _stream(stream))
    _check(rc, "dg_fp8_grouped_gemm_masked")


# ---------------------------------------------------------------------------
# MXFP4 and the mixture-of-experts layer
# ---------------------------------------------------------------------------

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def mxfp4_shapes(rows: int, cols: int):
    """(shape of the codes, shape of the scale words) of rows x cols values."""
    return (rows, cdiv(cols, 32) * 16), (cdiv(cols, 128), rows)


def _mxfp4_matrix(q, what):
    """(rows, values a row) of a matrix of codes."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if q.dim() != 2:
        raise ValueError("%s must be a matrix of codes" % what)
    return q.shape[0], 2 * q.shape[1]


def _mxfp4_pair(q, sf, rows, cols, what):
    _require(q, torch.uint8, what)
    _require(sf, torch.int32, "scales of " + what)
    if q.shape != (rows, (cols + 31) // 32 * 16) or sf.shape != ((cols + 127) // 128, rows):
        raise ValueError("%s must be codes %s and scales %s" % ((what,) + mxfp4_shapes(rows, cols)))


def _mxfp4_source(x):
    """(rows, cols, row stride, dtype code) of a matrix to quantise."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError("x must be a float32 or bfloat16 tensor")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    rows, cols = x.shape
    ld, one = x.stride()
    if cols > 1 and one != 1 or rows > 1 and ld < cols:
        raise ValueError("the rows of x must be contiguous and must not overlap")
    return rows, cols, ld if rows > 1 else cols, _DTYPES[x.dtype]


def dg_quantize_mxfp4(x, q=None, sf=None, qt=None, sft=None, stream=None) -> None:
    """x float32 or bfloat16 [rows, cols], its rows contiguous (any row stride)
    -> MXFP4 codes and scales along the rows (q, sf), along the columns (qt,
    sft: those of x.t()), or both; shapes as mxfp4_shapes gives them."""
    rows, cols, ld, dtype = _mxfp4_source(x)
    if q is not None or sf is not None:
        _mxfp4_pair(q, sf, rows, cols, "q")
    if qt is not None or sft is not None:
        _mxfp4_pair(qt, sft, cols, rows, "qt")
    _check(lib.dg_quantize_mxfp4(_ptr(q), _ptr(sf), _ptr(qt), _ptr(sft), _ptr(x), dtype, rows,
                                 cols, ld, _stream(stream)), "dg_quantize_mxfp4")


def dg_dequantize_mxfp4(out, q, sf, stream=None) -> None:
    """out [rows, cols] (float32 or bfloat16) = the values of codes q, sf."""
    if not isinstance(out, torch.Tensor) or out.dtype not in _DTYPES:
        raise TypeError("out must be a float32 or bfloat16 tensor")
    _require(out, out.dtype, "out")
    rows, cols = out.shape
    _mxfp4_pair(q, sf, rows, cols, "q")
    _check(lib.dg_dequantize_mxfp4(_ptr(out), _DTYPES[out.dtype], _ptr(q), _ptr(sf), rows, cols,
                                   _stream(stream)), "dg_dequantize_mxfp4")


def dg_mxfp4_gemm_nt_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.dg_mxfp4_gemm_nt_workspace_bytes(M, N, K)


def dg_mxfp4_gemm_nt(c, a, b, sfa, sfb, workspace=None, stream=None) -> None:
    """C[M,N] (bf16) = A . B^T, both MXFP4 (codes [M, K/2] and [N, K/2])."""
    c = _bf16(c, "c")
    M, N = c.shape
    rows, K = _mxfp4_matrix(a, "a")
    if rows != M or _mxfp4_matrix(b, "b") != (N, K):
        raise ValueError("shape mismatch: a %s, b %s, c %s" % (tuple(a.shape), tuple(b.shape),
                                                              tuple(c.shape)))
    _mxfp4_pair(a, sfa, M, K, "a")
    _mxfp4_pair(b, sfb, N, K, "b")
    _check(lib.dg_mxfp4_gemm_nt(_ptr(c), _ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb), M, N, K,
                                _ptr(workspace), _workspace_bytes(workspace), _stream(stream)),
           "dg_mxfp4_gemm_nt")


MXFP4_BF16A_MAX_M = 64


def dg_mxfp4_gemm_nt_bf16a_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.dg_mxfp4_gemm_nt_bf16a_workspace_bytes(M, N, K)


def dg_mxfp4_gemm_nt_bf16a(c, a, b, sfb, workspace=None, stream=None) -> None:
    """C[M,N] (bf16) = A[M,K] (bf16, not quantised) . B[N,K]^T (MXFP4);
    M <= MXFP4_BF16A_MAX_M."""
    c = _bf16(c, "c")
    a = _bf16(a, "a")
    M, K = a.shape
    N, per_row = _mxfp4_matrix(b, "b")
    if per_row != K or c.shape != (M, N):
        raise ValueError("shape mismatch: a %s, b %s, c %s" % (tuple(a.shape), tuple(b.shape),
                                                              tuple(c.shape)))
    _mxfp4_pair(b, sfb, N, K, "b")
    _check(lib.dg_mxfp4_gemm_nt_bf16a(_ptr(c), _ptr(a), _ptr(b), _ptr(sfb), M, N, K,
                                      _ptr(workspace), _workspace_bytes(workspace),
                                      _stream(stream)), "dg_mxfp4_gemm_nt_bf16a")


MOE_SCORINGS = {"softmax": 0, "sigmoid": 1}


def dg_moe_layer_workspace_bytes(T: int, E: int, k: int, H: int, I: int) -> int:
    return lib.dg_moe_layer_workspace_bytes(T, E, k, H, I)


def dg_moe_layer(y, x, w13, w2, s13, s2, ids, weights, logits=None, scoring: str = "softmax",
                 workspace=None, stream=None) -> None:
    """y [T,H] (bf16) = the mixture-of-experts layer on x [T,H] (bf16), T <=
    64.  w13 [E, 2I, H] (row 2i gate, 2i+1 up), w2 [E, H, I]: MXFP4 codes
    (uint8, two a byte, int32 scales [E, ceil(H/128), 2I] and [E, ceil(I/128),
    H]) or E4M3 (uint8 / float8_e4m3fn, float32 scales [E, H/128,
    ceil(2I/128)] and [E, I/128, ceil(H/128)]); the scales' type tells which.
    With logits float32 [T, E], ids int32 [T, k] and weights float32 [T, k]
    are outputs (the top k and their normalised scores); without, inputs.
    workspace: dg_moe_layer_workspace_bytes(T, E, k, H, I) bytes."""
    y = _bf16(y, "y")
    x = _bf16(x, "x")
    w13 = _codes(w13, "w13")
    w2 = _codes(w2, "w2")
    if not isinstance(s13, torch.Tensor) or s13.dtype not in (torch.int32, torch.float32):
        raise TypeError("s13 must be int32 (MXFP4) or float32 (E4M3)")
    fp8 = s13.dtype == torch.float32
    _require(s13, s13.dtype, "s13")
    _require(s2, s13.dtype, "s2")
    _require(ids, torch.int32, "ids")
    _require(weights, torch.float32, "weights")
    if w13.dim() != 3 or ids.dim() != 2:
        raise ValueError("w13 must be [E, 2I, ..] and ids [T, k]")
    T, H = x.shape
    E = w13.shape[0]
    I = w13.shape[1] // 2
    k = ids.shape[1]
    per = 1 if fp8 else 2
    scales = (((E, cdiv(H, 128), cdiv(2 * I, 128)), (E, cdiv(I, 128), cdiv(H, 128))) if fp8 else
              ((E, cdiv(H, 128), 2 * I), (E, cdiv(I, 128), H)))
    if (y.shape != x.shape or w13.shape != (E, 2 * I, H // per) or w2.shape != (E, H, I // per)
            or ids.shape != (T, k) or weights.shape != (T, k)
            or (tuple(s13.shape), tuple(s2.shape)) != scales):
        raise ValueError("inconsistent mixture-of-experts shapes")
    if logits is not None:
        _require(logits, torch.float32, "logits")
        if logits.shape != (T, E):
            raise ValueError("logits must be [T, E]")
    _check(lib.dg_moe_layer(_ptr(y), _ptr(x), _ptr(w13), _ptr(w2), _ptr(s13), _ptr(s2), int(fp8),
                            _ptr(ids), _ptr(weights), _ptr(logits), MOE_SCORINGS[scoring], T, E, k,
                            H, I, _ptr(workspace), _workspace_bytes(workspace), _stream(stream)),
           "dg_moe_layer")


# ---------------------------------------------------------------------------
# Around the grouped products: routing, layout, dispatch, combine, SwiGLU
# ---------------------------------------------------------------------------

# A launch takes less time than the checks of its tensors one by one, so each
# call first looks at all of them in one expression; only where that fails do
# the _refuse_ functions look again, for the reason to raise.

_CODES = (torch.uint8, torch.float8_e4m3fn)
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_device_now = torch._C._cuda_getDevice
_stream_now = torch._C._cuda_getCurrentRawStream


def _need(t, dtypes, shape, device, name):
    """t is a contiguous tensor of one of dtypes, of this shape (None: any),
    on device number `device`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(map(str, dtypes)), t.dtype))
    _require(t, t.dtype, name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != device:
        raise ValueError("%s is on device %d, other tensors on %d" % (name, t.get_device(), device))


def _need_fp8(q, s, rows, cols, device, name):
    """Codes [rows, cols] and their 1 x 128 scales."""
    _need(q, _CODES, (rows, cols), device, name)
    _need(s, (_F32,), ((cols + 127) // 128, rows), device, "scales of " + name)


def _is_fp8(q, s, rows, cols, device):
    return (q.dtype in _CODES and q.shape == (rows, cols) and q.get_device() == device
            and q.is_contiguous() and s.dtype is _F32 and s.shape == ((cols + 127) // 128, rows)
            and s.get_device() == device and s.is_contiguous())


def _need_rows(x, dtypes, name):
    """(rows, columns, row stride, device number) of a device matrix with
    contiguous rows of any stride."""
    try:
        (rows, cols), (ld, one), device = x.shape, x.stride(), x.get_device()
        if x.dtype in dtypes and device >= 0 and (one == 1 or cols <= 1) and (ld >= cols or rows <= 1):
            return rows, cols, ld if rows > 1 else cols, device
    except (AttributeError, ValueError):
        pass
    if not isinstance(x, torch.Tensor) or x.dtype not in dtypes:
        raise TypeError("%s must be a tensor of %s" % (name, " or ".join(map(str, dtypes))))
    if x.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    if not x.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    raise ValueError("the rows of %s must be contiguous and must not overlap" % name)


def _need_matrix(t, name):
    """The shape of a matrix whose type and place are looked at elsewhere."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    return t.shape


def _launch_stream(stream, device):
    """The stream of a launch, which goes to the current device: the tensors
    have to be there."""
    if device != _device_now():
        raise ValueError("the tensors are on device %d, the current one is %d"
                         % (device, _device_now()))
    return _stream_now(device) if stream is None else stream


def _scratch(workspace, device):
    """(address, bytes) of a workspace or of none."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor on device %d" % device)
    return workspace.data_ptr(), workspace.nbytes


def _refuse_slots(ids, weights, T, dev, name):
    k = _need_matrix(ids, name)[1]
    _need(ids, (_I32,), (T, k), dev, name)
    if weights is not None:
        _need(weights, (_F32,), (T, k), dev, "weights")


def dg_moe_route(ids, weights, logits, bias=None, scoring: str = "softmax", groups: int = 1,
                 top_groups=None, group_best: int = 1, renormalise: bool = True,
                 scale: float = 1.0, stream=None) -> None:
    """ids int32 [T, k], weights float32 [T, k] = the k experts of each token
    and their weights from logits [T, E] (float32 or bfloat16, any row
    stride).  bias float32 [E] is added to the scores for the choice alone;
    of `groups` groups of experts the top_groups (default: all) with the
    largest sums of their group_best largest choice values stay."""
    T, E, ld, dev = _need_rows(logits, _DTYPES, "logits")
    try:
        shape = ids.shape
        k = shape[1]
        ok = (shape[0] == T and weights.shape == shape and ids.dtype is _I32
              and weights.dtype is _F32 and ids.get_device() == dev == weights.get_device()
              and len(shape) == 2 and ids.is_contiguous() and weights.is_contiguous()
              and (bias is None or bias.dtype is _F32 and bias.shape == (E,)
                   and bias.get_device() == dev and bias.is_contiguous()))
    except (AttributeError, IndexError):
        ok = False
    if not ok:
        _refuse_slots(ids, None, T, dev, "ids")
        _need(weights, (_F32,), ids.shape, dev, "weights")
        _need(bias, (_F32,), (E,), dev, "bias")
    rc = lib.dg_moe_route(ids.data_ptr(), weights.data_ptr(), logits.data_ptr(),
                          _DTYPES[logits.dtype], ld, None if bias is None else bias.data_ptr(),
                          MOE_SCORINGS[scoring], groups,
                          groups if top_groups is None else top_groups, group_best,
                          bool(renormalise), scale, T, E, k, _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_moe_route")


def dg_moe_route_backward(dlogits, dweights, ids, logits, scoring: str = "softmax",
                          renormalise: bool = True, scale: float = 1.0, stream=None) -> None:
    """dlogits [T, E] (the type of logits, any row stride) from dweights
    float32 [T, k] and the forward call's ids, logits and settings."""
    T, E, ld, dev = _need_rows(logits, _DTYPES, "logits")
    rows, cols, ldd, where = _need_rows(dlogits, (logits.dtype,), "dlogits")
    if (rows, cols, where) != (T, E, dev):
        raise ValueError("dlogits must be [T, E] on the device of logits")
    try:
        shape = ids.shape
        k = shape[1]
        ok = (shape[0] == T and dweights.shape == shape and ids.dtype is _I32
              and dweights.dtype is _F32 and ids.get_device() == dev == dweights.get_device()
              and len(shape) == 2 and ids.is_contiguous() and dweights.is_contiguous())
    except (AttributeError, IndexError):
        ok = False
    if not ok:
        _refuse_slots(ids, None, T, dev, "ids")
        _need(dweights, (_F32,), ids.shape, dev, "dweights")
    rc = lib.dg_moe_route_backward(dlogits.data_ptr(), ldd, dweights.data_ptr(), ids.data_ptr(),
                                   logits.data_ptr(), _DTYPES[logits.dtype], ld,
                                   MOE_SCORINGS[scoring], bool(renormalise), scale, T, E, k,
                                   _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_moe_route_backward")


def dg_moe_plan_rows(T: int, E: int, k: int) -> int:
    return lib.dg_moe_plan_rows(T, E, k)


def dg_moe_plan_workspace_bytes(T: int, E: int, k: int) -> int:
    return lib.dg_moe_plan_workspace_bytes(T, E, k)


def dg_moe_plan(rows, pairs, m_indices, offsets, counts, ids, workspace=None, stream=None) -> None:
    """The grouped products' layout from ids int32 [T, k] (the experts of each
    token, < 0 or >= E: none): rows int32 [T, k], pairs and m_indices int32 [M],
    offsets int64 [E + 1], counts int32 [E]; M a multiple of 128, at least
    dg_moe_plan_rows(T, E, k).  workspace: dg_moe_plan_workspace_bytes(T, E, k)
    bytes of any contents."""
    try:
        T, k = shape = ids.shape
        dev, M, E = ids.get_device(), pairs.numel(), counts.numel()
        ok = (ids.dtype is rows.dtype is pairs.dtype is m_indices.dtype is counts.dtype is _I32
              and offsets.dtype is _I64 and rows.shape == shape and pairs.dim() == 1
              and counts.dim() == 1 and m_indices.shape == (M,) and offsets.shape == (E + 1,)
              and rows.get_device() == pairs.get_device() == m_indices.get_device()
              == offsets.get_device() == counts.get_device() == dev >= 0
              and ids.is_contiguous() and rows.is_contiguous() and pairs.is_contiguous()
              and m_indices.is_contiguous() and offsets.is_contiguous() and counts.is_contiguous())
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        shape = _need_matrix(ids, "ids")
        dev = ids.get_device()
        for t, n in ((ids, "ids"), (pairs, "pairs"), (counts, "counts")):
            _need(t, (_I32,), None, dev, n)
        _need(rows, (_I32,), shape, dev, "rows")
        _need(m_indices, (_I32,), (pairs.numel(),), dev, "m_indices")
        _need(offsets, (_I64,), (counts.numel() + 1,), dev, "offsets")
        raise ValueError("pairs and counts must have one dimension")
    rc = lib.dg_moe_plan(rows.data_ptr(), pairs.data_ptr(), m_indices.data_ptr(),
                         offsets.data_ptr(), counts.data_ptr(), ids.data_ptr(), T, E, k, M,
                         *_scratch(workspace, dev), _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_moe_plan")


def dg_moe_dispatch_fp8_workspace_bytes(T: int, k: int, H: int, weighted: bool = False) -> int:
    return lib.dg_moe_dispatch_fp8_workspace_bytes(T, k, H, bool(weighted))


def _dispatch_workspace(workspace, stream, T, k, H, weights, device):
    """The caller's workspace, else one from torch for a call that has use for
    it; torch's memory belongs to its current stream, so not where the call
    is sent to another one."""
    if workspace is not None or stream is not None or T * k * H < 1 << 26:
        return workspace  # that few have no use for one: the library is asked about the others
    n = lib.dg_moe_dispatch_fp8_workspace_bytes(T, k, H, weights is not None)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _are_slots(rows, weights, T, device):
    shape = rows.shape
    return (rows.dtype is _I32 and len(shape) == 2 and shape[0] == T
            and rows.get_device() == device and rows.is_contiguous()
            and (weights is None or weights.dtype is _F32 and weights.shape == shape
                 and weights.get_device() == device and weights.is_contiguous()))


def dg_moe_dispatch_fp8(a, sa, x, rows, pairs, weights=None, workspace=None, stream=None) -> None:
    """a (codes [M, H]) and sa float32 [H/128, M] = the rows of x [T, H]
    (float32 or bfloat16, any row stride), times weights float32 [T, k] if
    given, quantised with 1 x 128 scales, at the rows of a dg_moe_plan.
    workspace: dg_moe_dispatch_fp8_workspace_bytes(T, k, H, weighted) bytes;
    without one, and without a stream, a large call takes its own from
    torch."""
    T, H, ld, dev = _need_rows(x, _DTYPES, "x")
    try:
        M = pairs.numel()
        ok = (pairs.dtype is _I32 and pairs.get_device() == dev and pairs.is_contiguous()
              and _are_slots(rows, weights, T, dev) and _is_fp8(a, sa, M, H, dev))
    except AttributeError:
        ok = False
    if not ok:
        _refuse_slots(rows, weights, T, dev, "rows")
        _need(pairs, (_I32,), None, dev, "pairs")
        _need_fp8(a, sa, pairs.numel(), H, dev, "a")
    k = rows.shape[1]
    workspace = _dispatch_workspace(workspace, stream, T, k, H, weights, x.device)
    rc = lib.dg_moe_dispatch_fp8(a.data_ptr(), sa.data_ptr(), x.data_ptr(), _DTYPES[x.dtype], ld,
                                 rows.data_ptr(), pairs.data_ptr(),
                                 None if weights is None else weights.data_ptr(), T, k, M, H,
                                 *_scratch(workspace, dev), _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_moe_dispatch_fp8")


def dg_moe_combine(y, c, rows, weights=None, residual=None, stream=None) -> None:
    """y [T, H] (bf16) = sum over the slots of weights (float32 [T, k], or all
    1) times the rows of c [M, H] (bf16), plus residual [T, H] (bf16)."""
    try:
        shape, slots, dev = y.shape, rows.shape, y.get_device()
        (T, H), (M, cols), k = shape, c.shape, slots[1]
        ok = (cols == H and slots[0] == T and len(slots) == 2 and y.dtype in _BF16_TYPES
              and c.dtype in _BF16_TYPES and rows.dtype is _I32
              and c.get_device() == rows.get_device() == dev >= 0
              and y.is_contiguous() and c.is_contiguous() and rows.is_contiguous()
              and (weights is None or weights.dtype is _F32 and weights.shape == slots
                   and weights.get_device() == dev and weights.is_contiguous())
              and (residual is None or residual.dtype in _BF16_TYPES and residual.shape == shape
                   and residual.get_device() == dev and residual.is_contiguous()))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        shape, (M, _) = _need_matrix(y, "y"), _need_matrix(c, "c")
        dev = y.get_device()
        _need(y, _BF16_TYPES, None, dev, "y")
        _need(c, _BF16_TYPES, (M, shape[1]), dev, "c")
        _refuse_slots(rows, weights, shape[0], dev, "rows")
        _need(residual, _BF16_TYPES, shape, dev, "residual")
    rc = lib.dg_moe_combine(y.data_ptr(), c.data_ptr(), rows.data_ptr(),
                            None if weights is None else weights.data_ptr(),
                            None if residual is None else residual.data_ptr(), T, k, M, H,
                            _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_moe_combine")


def dg_moe_combine_backward(dc, sdc, dweights, dy, c, rows, pairs, weights=None, workspace=None,
                            stream=None) -> None:
    """From dy [T, H] (bf16, any row stride): dc (codes [M, H]) and sdc float32
    [H/128, M], the gradient of c quantised as dg_moe_dispatch_fp8 does with
    weights, and dweights float32 [T, k]; dc and sdc, or dweights, may be
    None.  workspace: as for dg_moe_dispatch_fp8."""
    T, H, ld, dev = _need_rows(dy, (torch.bfloat16,), "dy")
    try:
        M = pairs.numel()
        ok = (pairs.dtype is _I32 and pairs.get_device() == dev and pairs.is_contiguous()
              and _are_slots(rows, weights, T, dev)
              and (dc is None and sdc is None or _is_fp8(dc, sdc, M, H, dev))
              and (dweights is None or _are_slots(rows, dweights, T, dev)
                   and c.dtype in _BF16_TYPES and c.shape == (M, H) and c.get_device() == dev
                   and c.is_contiguous()))
    except AttributeError:
        ok = False
    if not ok:
        _refuse_slots(rows, weights, T, dev, "rows")
        _need(pairs, (_I32,), None, dev, "pairs")
        M = pairs.numel()
        if dc is not None or sdc is not None:
            _need_fp8(dc, sdc, M, H, dev, "dc")
        _need(dweights, (_F32,), rows.shape, dev, "dweights")
        _need(c, _BF16_TYPES, (M, H), dev, "c")
    k = rows.shape[1]
    if dc is not None:
        workspace = _dispatch_workspace(workspace, stream, T, k, H, weights, dy.device)
    rc = lib.dg_moe_combine_backward(None if dc is None else dc.data_ptr(),
                                     None if dc is None else sdc.data_ptr(),
                                     None if dweights is None else dweights.data_ptr(),
                                     dy.data_ptr(), ld, None if dweights is None else c.data_ptr(),
                                     rows.data_ptr(), pairs.data_ptr(),
                                     None if weights is None else weights.data_ptr(), T, k, M, H,
                                     *_scratch(workspace, dev), _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_moe_combine_backward")


def _are_layout_rows(m_indices, M, device):
    return m_indices is None or (m_indices.dtype is _I32 and m_indices.shape == (M,)
                                 and m_indices.get_device() == device
                                 and m_indices.is_contiguous())


def dg_swiglu_fp8(h, sh, gu, kept=None, skept=None, m_indices=None, stream=None) -> None:
    """h (codes [M, I]) and sh float32 [I/128, M] = silu(gate) * up of gu [M, 2I]
    (bf16, column 2i gate, 2i+1 up), and kept (codes [M, 2I]), skept float32
    [2I/128, M] = gu itself in 8 bits for dg_swiglu_fp8_backward.  m_indices
    int32 [M]: the rows of the grouped layout that are real."""
    M, two = _need_matrix(gu, "gu")
    dev = gu.get_device()
    try:
        ok = (two % 2 == 0 and gu.dtype in _BF16_TYPES and dev >= 0 and gu.is_contiguous()
              and _is_fp8(h, sh, M, two // 2, dev) and _are_layout_rows(m_indices, M, dev)
              and (kept is None and skept is None or _is_fp8(kept, skept, M, two, dev)))
    except AttributeError:
        ok = False
    if not ok:
        _need(gu, _BF16_TYPES, None, dev, "gu")
        if two % 2:
            raise ValueError("gu must be [M, 2I]")
        _need_fp8(h, sh, M, two // 2, dev, "h")
        if kept is not None or skept is not None:
            _need_fp8(kept, skept, M, two, dev, "kept")
        _need(m_indices, (_I32,), (M,), dev, "m_indices")
    rc = lib.dg_swiglu_fp8(h.data_ptr(), sh.data_ptr(), None if kept is None else kept.data_ptr(),
                           None if kept is None else skept.data_ptr(), gu.data_ptr(),
                           None if m_indices is None else m_indices.data_ptr(), M, two // 2,
                           _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_swiglu_fp8")


def dg_swiglu_fp8_backward(dgu, sdgu, dh, kept, skept, h=None, sh=None, m_indices=None,
                           stream=None) -> None:
    """dgu (codes [M, 2I]) and sdgu from dh [M, I] (bf16) and the checkpoint
    kept, skept; with h (codes [M, I]) and sh also silu(gate) * up of the
    checkpoint's values."""
    M, I = _need_matrix(dh, "dh")
    dev = dh.get_device()
    try:
        ok = (dh.dtype in _BF16_TYPES and dev >= 0 and dh.is_contiguous()
              and _is_fp8(dgu, sdgu, M, 2 * I, dev) and _is_fp8(kept, skept, M, 2 * I, dev)
              and (h is None and sh is None or _is_fp8(h, sh, M, I, dev))
              and _are_layout_rows(m_indices, M, dev))
    except AttributeError:
        ok = False
    if not ok:
        _need(dh, _BF16_TYPES, None, dev, "dh")
        _need_fp8(dgu, sdgu, M, 2 * I, dev, "dgu")
        _need_fp8(kept, skept, M, 2 * I, dev, "kept")
        if h is not None or sh is not None:
            _need_fp8(h, sh, M, I, dev, "h")
        _need(m_indices, (_I32,), (M,), dev, "m_indices")
    rc = lib.dg_swiglu_fp8_backward(dgu.data_ptr(), sdgu.data_ptr(),
                                    None if h is None else h.data_ptr(),
                                    None if h is None else sh.data_ptr(), dh.data_ptr(),
                                    kept.data_ptr(), skept.data_ptr(),
                                    None if m_indices is None else m_indices.data_ptr(), M, I,
                                    _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_swiglu_fp8_backward")


def dg_transpose_fp8_blocks(qt, st, q, s, block_rows: int = 128, m_indices=None,
                            stream=None) -> None:
    """qt (codes [C, M]) and st float32 [M/128, C] (block_rows 1) or [M/128,
    C/128] (block_rows 128) = the transpose of q (codes [M, C], 1 x 128 scales
    s float32 [C/128, M]), quantised anew along the rows of q."""
    M, C = _need_matrix(q, "q")
    dev, blocks = q.get_device(), ((M + 127) // 128, C if block_rows == 1 else (C + 127) // 128)
    try:
        ok = (dev >= 0 and _is_fp8(q, s, M, C, dev) and qt.dtype in _CODES and qt.shape == (C, M)
              and qt.get_device() == dev and qt.is_contiguous() and st.dtype is _F32
              and st.shape == blocks and st.get_device() == dev and st.is_contiguous()
              and _are_layout_rows(m_indices, M, dev))
    except AttributeError:
        ok = False
    if not ok:
        _need_fp8(q, s, M, C, dev, "q")
        _need(qt, _CODES, (C, M), dev, "qt")
        _need(st, (_F32,), blocks, dev, "st")
        _need(m_indices, (_I32,), (M,), dev, "m_indices")
    rc = lib.dg_transpose_fp8_blocks(qt.data_ptr(), st.data_ptr(), block_rows, q.data_ptr(),
                                     s.data_ptr(),
                                     None if m_indices is None else m_indices.data_ptr(), M, C,
                                     _launch_stream(stream, dev))
    if rc:
        raise DGError(rc, "dg_transpose_fp8_blocks")


# ---------------------------------------------------------------------------
# Conveniences (allocate outputs with torch)
# ---------------------------------------------------------------------------

def to_fp8(x, block_rows: int = 128):
    """Quantise a float32 device matrix -> (codes uint8 [R, C], scales float32
    [ceil(C/128), ceil(R/block_rows)])."""
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    s = torch.empty((cdiv(cols, 128), cdiv(rows, block_rows)), dtype=torch.float32,
                    device=x.device)
    dg_quantize_fp8_block(q, s, x, block_rows)
    return q, s


def to_fp8_ue8m0(x, block_rows: int = 128):
    """Quantise with power-of-two scales -> (codes uint8 [R, C], packed UE8M0
    exponents int32 [ceil(C/512), ceil(R/block_rows)])."""
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    sf = torch.empty((cdiv(cdiv(cols, 128), 4), cdiv(rows, block_rows)), dtype=torch.int32,
                     device=x.device)
    dg_quantize_fp8_block_ue8m0(q, sf, x, block_rows)
    return q, sf


def fp8_gemm_nt(c, a, b, sa, sb, a_block_rows: int = 128, workspace=None):
    dg_fp8_gemm_nt(c, a, b, sa, sb, a_block_rows, workspace)
    return c


def fp8_grouped_gemm_contig(c, a, b, sa, sb, m_indices, a_block_rows: int = 1):
    dg_fp8_grouped_gemm_contig(c, a, b, sa, sb, a_block_rows, m_indices, workspace=None)
    return c


def _mxfp4_empty(rows, cols, device):
    qs, ss = mxfp4_shapes(rows, cols)
    return (torch.empty(qs, dtype=torch.uint8, device=device),
            torch.empty(ss, dtype=torch.int32, device=device))


def to_mxfp4(x, transposed: bool = False):
    """Quantise a float32 or bfloat16 device matrix to MXFP4 along its rows,
    or (transposed) along its columns -> (codes, scales) of x, or of x.t()."""
    rows, cols, ld, dtype = _mxfp4_source(x)
    q, sf = _mxfp4_empty(cols, rows, x.device) if transposed else _mxfp4_empty(rows, cols, x.device)
    p = q.data_ptr(), sf.data_ptr()
    p = (None, None) + p if transposed else p + (None, None)
    _check(lib.dg_quantize_mxfp4(*p, x.data_ptr(), dtype, rows, cols, ld, _stream(None)),
           "dg_quantize_mxfp4")
    return q, sf


def to_mxfp4_both(x):
    """Both directions from one reading of x: (q, sf) of x, (qt, sft) of
    x.t()."""
    rows, cols, ld, dtype = _mxfp4_source(x)
    q, sf = _mxfp4_empty(rows, cols, x.device)
    qt, sft = _mxfp4_empty(cols, rows, x.device)
    _check(lib.dg_quantize_mxfp4(q.data_ptr(), sf.data_ptr(), qt.data_ptr(), sft.data_ptr(),
                                 x.data_ptr(), dtype, rows, cols, ld, _stream(None)),
           "dg_quantize_mxfp4")
    return q, sf, qt, sft


def from_mxfp4(q, sf, cols: int, dtype=torch.bfloat16):
    """The values [rows, cols] of MXFP4 codes q and scales sf."""
    out = torch.empty((_mxfp4_matrix(q, "q")[0], cols), dtype=dtype, device=q.device)
    dg_dequantize_mxfp4(out, q, sf)
    return out


def mxfp4_gemm_nt(a, b, sfa, sfb, workspace=None):
    """A . B^T of two MXFP4 matrices -> bfloat16 [M, N]."""
    M, N = _mxfp4_matrix(a, "a")[0], _mxfp4_matrix(b, "b")[0]
    c = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    dg_mxfp4_gemm_nt(c, a, b, sfa, sfb, workspace)
    return c


def moe_route(logits, k: int, bias=None, scoring: str = "softmax", groups: int = 1,
              top_groups=None, group_best: int = 1, renormalise: bool = True, scale: float = 1.0):
    """The k experts of each token and their weights: int32, float32 [T, k]."""
    T = logits.shape[0]
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    dg_moe_route(ids, weights, logits, bias, scoring, groups, top_groups, group_best, renormalise,
                 scale)
    return ids, weights


#: The layout that dg_moe_plan writes.
MoePlan = collections.namedtuple("MoePlan", "rows pairs m_indices offsets counts")


def moe_plan(ids, experts: int):
    """The grouped products' layout of the experts ids int32 [T, k]."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise TypeError("ids must be an int32 tensor [T, k]")
    T, k = ids.shape
    M, n = dg_moe_plan_rows(T, experts, k), dg_moe_plan_workspace_bytes(T, experts, k)
    if M == 0:
        raise ValueError("no layout for %d tokens, %d experts, %d slots" % (T, experts, k))
    new = dict(dtype=torch.int32, device=ids.device)
    plan = MoePlan(torch.empty((T, k), **new), torch.empty(M, **new), torch.empty(M, **new),
                   torch.empty(experts + 1, dtype=torch.int64, device=ids.device),
                   torch.empty(experts, **new))
    ws = torch.empty(n, dtype=torch.uint8, device=ids.device) if n else None
    dg_moe_plan(*plan, ids, workspace=ws)
    return plan


def _fp8_empty(rows, cols, device):
    return (torch.empty((rows, cols), dtype=torch.uint8, device=device),
            torch.empty((cdiv(cols, 128), rows), dtype=torch.float32, device=device))


def moe_dispatch_fp8(x, plan, weights=None):
    """x [T, H] into the layout -> (codes [M, H], scales [H/128, M]).  Blocks
    of 128 rows without an expert keep what the memory held."""
    a, sa = _fp8_empty(plan.pairs.numel(), x.shape[1], x.device)
    dg_moe_dispatch_fp8(a, sa, x, plan.rows, plan.pairs, weights)
    return a, sa


def moe_combine(c, plan, weights=None, residual=None):
    """The rows c [M, H] of the layout summed per token -> bfloat16 [T, H]."""
    y = torch.empty((plan.rows.shape[0], c.shape[1]), dtype=torch.bfloat16, device=c.device)
    dg_moe_combine(y, c, plan.rows, weights, residual)
    return y


def swiglu_fp8(gu, m_indices=None, keep: bool = False):
    """silu(gate) * up of gu [M, 2I] -> (codes [M, I], scales [I/128, M]), and
    with keep the checkpoint (codes [M, 2I], scales) after them."""
    M, two = gu.shape
    h, sh = _fp8_empty(M, two // 2, gu.device)
    kept, skept = _fp8_empty(M, two, gu.device) if keep else (None, None)
    dg_swiglu_fp8(h, sh, gu, kept, skept, m_indices)
    return (h, sh, kept, skept) if keep else (h, sh)


def transpose_fp8_blocks(q, s, block_rows: int = 128, m_indices=None):
    """Codes [M, C] with 1 x 128 scales -> (codes [C, M], scales over 128 rows
    of one column (block_rows 1) or of 128)."""
    M, C = q.shape
    qt = torch.empty((C, M), dtype=torch.uint8, device=q.device)
    st = torch.empty((cdiv(M, 128), C if block_rows == 1 else cdiv(C, 128)), dtype=torch.float32,
                     device=q.device)
    dg_transpose_fp8_blocks(qt, st, q, s, block_rows, m_indices)
    return qt, st


__all__ = [
    "lib", "LIB_PATH", "DGError", "status_string", "get_mk_alignment_for_contiguous_layout",
    "dg_quantize_fp8_block", "dg_fp8_gemm_nt_workspace_bytes", "dg_fp8_gemm_nt",
    "dg_fp8_gemm_nt_fused_a", "FUSED_A_MAX_M", "dg_fp8_grouped_gemm_contig", "to_fp8",
    "dg_quantize_fp8_block_ue8m0", "dg_fp8_gemm_nt_ue8m0", "to_fp8_ue8m0",
    "dg_fp8_gemm_nt_epilogue", "EPILOGUES", "dg_transpose_fp8", "dg_fp8_gemm_workspace_bytes",
    "dg_fp8_gemm", "LAYOUTS", "dg_fp8_grouped_gemm_k", "fp8_gemm_nt", "fp8_grouped_gemm_contig",
    "dg_fp8_grouped_gemm_masked", "dg_fp8_grouped_gemm_masked_workspace_bytes",
    "dg_fp8_grouped_gemm_contig_ue8m0", "dg_fp8_grouped_gemm_masked_ue8m0", "alloc_workspace",
    "WORKSPACE_COUNTER_BYTES", "dg_fp8_gemm_nt_noalloc", "NOALLOC_SCRATCH_BYTES",
    "mxfp4_shapes", "dg_quantize_mxfp4", "dg_dequantize_mxfp4", "to_mxfp4", "to_mxfp4_both",
    "from_mxfp4", "dg_mxfp4_gemm_nt_workspace_bytes", "dg_mxfp4_gemm_nt", "mxfp4_gemm_nt",
    "dg_mxfp4_gemm_nt_bf16a_workspace_bytes", "dg_mxfp4_gemm_nt_bf16a", "MXFP4_BF16A_MAX_M",
    "dg_moe_layer_workspace_bytes", "dg_moe_layer", "MOE_SCORINGS",
    "dg_moe_route", "dg_moe_route_backward", "moe_route", "dg_moe_plan_rows",
    "dg_moe_plan_workspace_bytes", "dg_moe_plan", "MoePlan", "moe_plan", "dg_moe_dispatch_fp8",
    "dg_moe_dispatch_fp8_workspace_bytes", "moe_dispatch_fp8", "dg_moe_combine", "dg_moe_combine_backward", "moe_combine",
    "dg_swiglu_fp8", "dg_swiglu_fp8_backward", "swiglu_fp8", "dg_transpose_fp8_blocks",
    "transpose_fp8_blocks",
]
# (the _epilogue C entry points are reached through the act / residual
# arguments of dg_fp8_grouped_gemm_contig and dg_fp8_grouped_gemm_masked)
