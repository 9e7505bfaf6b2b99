"""Thin Python binding of the NVFP4 C ABI (include/nvfp4.h, include/nvfp4_ffn.h).

Argument marshalling only: every entry point takes torch CUDA tensors, passes
their data pointers and the current CUDA stream to the function of the same
name in libnvfp4.so, and raises on a non-zero status. All arithmetic runs in
the library's kernels; there is no fallback of any kind. Output tensors and
workspaces are allocated here with torch (the library itself never allocates).
Every call takes `stream`: the torch.cuda.Stream to run on, the current one by default; what the call
allocates belongs to that stream, and the caller orders it against other streams as any torch work.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libnvfp4.so")

NVFP4_TUNE_DENSE_BN = 1
NVFP4_TUNE_DENSE_GRID = 2
NVFP4_TUNE_STREAM_MAX_M = 3
NVFP4_TUNE_STREAM_SPLIT = 4
NVFP4_TUNE_STREAM_STAGES = 5
NVFP4_TUNE_GROUPED_GRID = 6
NVFP4_TUNE_GROUPED_STAGES = 7
NVFP4_TUNE_DENSE_KERNEL = 8
NVFP4_TUNE_PDL = 9
NVFP4_TUNE_WEIGHT_L2 = 10
NVFP4_TUNE_DENSE_RASTER = 11
NVFP4_TUNE_WATCHDOG_US = 12
NVFP4_TUNE_TEST_WITHHOLD_STAGE = 13
NVFP4_TUNE_STREAM_L2_PREFETCH = 14
NVFP4_TUNE_GROUPED_TILE_ROWS = 15

STATUS = {0: "NVFP4_OK", -1: "NVFP4_ERR_INVALID_ARG", -2: "NVFP4_ERR_UNSUPPORTED_SHAPE",
          -3: "NVFP4_ERR_ALIGNMENT", -4: "NVFP4_ERR_ARCH", -5: "NVFP4_ERR_CUDA",
          -6: "NVFP4_ERR_WORKSPACE", -7: "NVFP4_ERR_TIMEOUT", -8: "NVFP4_ERR_BAD_OFFSETS"}

EXPORTS = ["nvfp4_status_string", "nvfp4_scale_bytes", "nvfp4_amax_workspace_bytes", "nvfp4_amax",
           "nvfp4_quantize", "nvfp4_gemm_workspace_bytes", "nvfp4_gemm", "nvfp4_gemm_quantize_out",
           "nvfp4_grouped_gemm_workspace_bytes", "nvfp4_grouped_gemm", "nvfp4_grouped_gemm_gather",
           "nvfp4_grouped_gemm_gather_workspace_bytes",
           "nvfp4_grouped_gemm_swiglu",
           "nvfp4_grouped_gemm_noalloc",
           "nvfp4_encode_e2m1",
           "nvfp4_encode_e4m3", "nvfp4_tune", "nvfp4_last_launch_count",
           "nvfp4_sparse_meta_bytes", "nvfp4_scale_bytes_b32", "nvfp4_prune_pairs", "nvfp4_quantize_b32",
           "nvfp4_sparse_gemm", "nvfp4_grouped_sparse_gemm", "nvfp4_gemm_batched",
           "nvfp4_grouped_gemm_swiglu_quantize_out",
           "nvfp4_moe_route_workspace_bytes", "nvfp4_moe_route", "nvfp4_moe_route_backward", "nvfp4_fp8_quantize",
           "nvfp4_fp8_gemm", "nvfp4_fp8_grouped_gemm_workspace_bytes", "nvfp4_fp8_grouped_gemm"]
# of include/nvfp4_ffn.h
EXPORTS_FFN = ["nvfp4_gated_ffn_workspace_bytes", "nvfp4_gated_ffn", "nvfp4_gated_ffn_backward_workspace_bytes",
               "nvfp4_gated_ffn_backward", "nvfp4_int8_quantize", "nvfp4_int8_gemm_workspace_bytes", "nvfp4_int8_gemm",
               "nvfp4_grad_clip_workspace_bytes", "nvfp4_grad_clip"]


class NVFP4Error(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")
        self.status = status


_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t

NVFP4_MAX_BATCH = 8


class GemmProblem(ctypes.Structure):
    """One problem of nvfp4_gemm_batched (the C struct nvfp4_gemm_problem)."""
    _fields_ = [("a", ctypes.c_void_p), ("sfa", ctypes.c_void_p), ("ga", ctypes.c_void_p),
                ("b", ctypes.c_void_p), ("sfb", ctypes.c_void_p), ("gb", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


def lib():
    """The loaded libnvfp4.so; raises if it was not built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"NVFP4 CUDA library missing at {LIB_PATH}: run "
                                  "`python -c 'import __graft_entry__ as g; g.build()'` first")
            L = ctypes.CDLL(LIB_PATH)
            L.nvfp4_status_string.restype = ctypes.c_char_p
            L.nvfp4_status_string.argtypes = [ctypes.c_int]
            L.nvfp4_scale_bytes.restype = _i64
            L.nvfp4_scale_bytes.argtypes = [_i64, _i64]
            L.nvfp4_amax_workspace_bytes.restype = _sz
            L.nvfp4_amax_workspace_bytes.argtypes = [_i64]
            L.nvfp4_amax.argtypes = [_vp, _i64, _vp, _vp, _vp, _sz, _vp]
            L.nvfp4_quantize.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _vp]
            L.nvfp4_gemm_workspace_bytes.restype = _sz
            L.nvfp4_gemm_workspace_bytes.argtypes = [_i64, _i64, _i64]
            L.nvfp4_gemm.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz,
                                     _vp, _vp]
            L.nvfp4_gemm_quantize_out.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                                  _i64, _vp, _vp]
            L.nvfp4_grouped_gemm_workspace_bytes.restype = _sz
            L.nvfp4_grouped_gemm_workspace_bytes.argtypes = [_i32, _i64, _i64, _i64]
            L.nvfp4_grouped_gemm.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64,
                                             _i64, _vp, _vp, _sz, _vp, _vp]
            L.nvfp4_grouped_gemm_gather_workspace_bytes.restype = _sz
            L.nvfp4_grouped_gemm_gather_workspace_bytes.argtypes = [_i32, _i64, _i64, _i64]
            L.nvfp4_grouped_gemm_gather.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64,
                                                    _i64, _i64, _vp, _vp, _sz, _vp, _vp]
            L.nvfp4_grouped_gemm_swiglu.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64,
                                                    _i64, _vp, _vp, _sz, _vp, _vp]
            L.nvfp4_grouped_gemm_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64,
                                                     _i64, _i64, _vp, _vp, _vp]
            L.nvfp4_encode_e2m1.argtypes = [_vp, _i64, _vp, _vp]
            L.nvfp4_encode_e4m3.argtypes = [_vp, _i64, _vp, _vp]
            L.nvfp4_tune.argtypes = [ctypes.c_int, ctypes.c_int]
            L.nvfp4_sparse_meta_bytes.restype = _i64
            L.nvfp4_sparse_meta_bytes.argtypes = [_i64, _i64]
            L.nvfp4_scale_bytes_b32.restype = _i64
            L.nvfp4_scale_bytes_b32.argtypes = [_i64, _i64]
            L.nvfp4_prune_pairs.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp]
            L.nvfp4_quantize_b32.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _vp]
            L.nvfp4_sparse_gemm.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]
            L.nvfp4_grouped_sparse_gemm.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64,
                                                    _i64, _vp, _vp, _sz, _vp, _vp]
            L.nvfp4_gemm_batched.argtypes = [_vp, _i32, _i64, _vp, _vp]
            L.nvfp4_grouped_gemm_swiglu_quantize_out.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64,
                                                                 _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
            L.nvfp4_moe_route_workspace_bytes.restype = _sz
            L.nvfp4_moe_route_workspace_bytes.argtypes = [_i64, _i32]
            L.nvfp4_moe_route.argtypes = [_vp, _i32, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _sz, _vp]
            L.nvfp4_moe_route_backward.argtypes = [_vp, _i32, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                                   _vp, _vp, _vp]
            L.nvfp4_fp8_quantize.argtypes = [_vp, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp]
            L.nvfp4_fp8_gemm.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp]
            L.nvfp4_fp8_grouped_gemm_workspace_bytes.restype = _sz
            L.nvfp4_fp8_grouped_gemm_workspace_bytes.argtypes = [_i32, _i64, _i64, _i64]
            L.nvfp4_fp8_grouped_gemm.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _sz, _vp,
                                                 _vp]
            L.nvfp4_gated_ffn_workspace_bytes.restype = _sz
            L.nvfp4_gated_ffn_workspace_bytes.argtypes = [_i64, _i64, _i64]
            L.nvfp4_gated_ffn.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _i64,
                                          _i64, _vp, _sz, _vp, _vp]
            L.nvfp4_gated_ffn_backward_workspace_bytes.restype = _sz
            L.nvfp4_gated_ffn_backward_workspace_bytes.argtypes = [_i64, _i64, _i64]
            L.nvfp4_gated_ffn_backward.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _vp,
                                                   _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp, _vp]
            L.nvfp4_int8_quantize.argtypes = [_vp, _i64, _i32, _i64, _i64, _vp, _vp, _vp]
            L.nvfp4_int8_gemm_workspace_bytes.restype = _sz
            L.nvfp4_int8_gemm_workspace_bytes.argtypes = [_i64, _i64, _i64]
            L.nvfp4_int8_gemm.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _sz, _vp, _vp]
            L.nvfp4_grad_clip_workspace_bytes.restype = _sz
            L.nvfp4_grad_clip_workspace_bytes.argtypes = [_i32]
            L.nvfp4_grad_clip.argtypes = [_vp, _vp, _vp, _vp, _i32, ctypes.c_float, _vp, _vp, _sz, _vp]
            L.nvfp4_last_launch_count.restype = ctypes.c_int
            _lib = L
    return _lib


def _ptr(t):  # an int: every entry point's argtypes convert it to the pointer
    if t is None:
        return None
    if not t.is_cuda:
        raise TypeError("operands must be CUDA tensors")
    return t.data_ptr()


def _status(t):
    """dev_status's address: None, or where the kernels write a status."""
    return None if t is None else _operand(t, _I32, (1,), "dev_status")


def _stream():
    # the current stream's handle without the Stream object (3 us of a small call's host time)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _on_stream(stream, fn, args):
    """The call fn(**args) with `stream` as the current stream, so that what it allocates (outputs, workspaces)
    is that stream's: torch's allocator then neither hands the call a block that another stream still reads nor
    passes a dropped workspace on while the kernels use it. The outputs are recorded for the caller's current
    stream too, where they are usually read next (after waiting)."""
    args["stream"] = None
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = fn(**args)
    if stream != here:
        for t in out if isinstance(out, tuple) else (out,):
            t = t._buf if isinstance(t, MoeRouting) else t
            if t is not None:
                t.record_stream(here)
    return out


def _check(fn, rc):
    if rc != 0:
        raise NVFP4Error(fn, rc)


def _cuda(t, dtype, name):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous CUDA tensor of {dtype}")
    return t


def nvfp4_scale_bytes(rows: int, K: int) -> int:
    return int(lib().nvfp4_scale_bytes(rows, K))


def nvfp4_tune(key: int, value: int) -> None:
    _check("nvfp4_tune", lib().nvfp4_tune(key, value))


def nvfp4_last_launch_count() -> int:
    return int(lib().nvfp4_last_launch_count())


def nvfp4_amax_workspace_bytes(n: int) -> int:
    return int(lib().nvfp4_amax_workspace_bytes(n))


def nvfp4_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().nvfp4_gemm_workspace_bytes(M, N, K))


def nvfp4_status_string(status: int) -> str:
    return lib().nvfp4_status_string(status).decode()


def nvfp4_amax(x: torch.Tensor, amax_out=None, g_out=None, workspace=None, stream=None):
    """Returns (amax, g) as 1-element fp32 CUDA tensors; g = amax / 2688 (1 if amax == 0)."""
    if stream is not None:
        return _on_stream(stream, nvfp4_amax, locals())
    _cuda(x, torch.bfloat16, "x")
    dev = x.device
    amax_out = torch.empty(1, dtype=torch.float32, device=dev) if amax_out is None else amax_out
    g_out = torch.empty(1, dtype=torch.float32, device=dev) if g_out is None else g_out
    nbytes = int(lib().nvfp4_amax_workspace_bytes(x.numel()))
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check("nvfp4_amax", lib().nvfp4_amax(_ptr(x), x.numel(), _ptr(amax_out), _ptr(g_out),
                                          _ptr(workspace), workspace.numel(), _stream()))
    return amax_out, g_out


def nvfp4_quantize(x: torch.Tensor, global_scale: torch.Tensor, q_out=None, sf_out=None, stream=None):
    """bf16 [M, K] -> (q u8 [M, K/2], sf u8 [nvfp4_scale_bytes(M, K)])."""
    if stream is not None:
        return _on_stream(stream, nvfp4_quantize, locals())
    _cuda(x, torch.bfloat16, "x")
    _cuda(global_scale, torch.float32, "global_scale")
    M, K = x.shape
    q_out = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device) if q_out is None else q_out
    sf_out = (torch.empty(nvfp4_scale_bytes(M, K), dtype=torch.uint8, device=x.device)
              if sf_out is None else sf_out)
    _check("nvfp4_quantize", lib().nvfp4_quantize(_ptr(x), M, K, _ptr(global_scale), _ptr(q_out),
                                                  _ptr(sf_out), _stream()))
    return q_out, sf_out


def nvfp4_gemm(a, sfa, ga, b, sfb, gb, M: int, N: int, K: int, y=None, dev_status=None,
               stream=None):
    """y = x @ W^T in bf16 [M, N] from packed NVFP4 operands (see include/nvfp4.h)."""
    if stream is not None:
        return _on_stream(stream, nvfp4_gemm, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b, "b"), (sfb, "sfb")):
        _cuda(t, torch.uint8, n)
    _cuda(ga, torch.float32, "ga")
    _cuda(gb, torch.float32, "gb")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=a.device) if y is None else y
    ws_bytes = int(lib().nvfp4_gemm_workspace_bytes(M, N, K))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=a.device) if ws_bytes else None
    _check("nvfp4_gemm", lib().nvfp4_gemm(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b), _ptr(sfb), _ptr(gb),
                                          _ptr(y), M, N, K, _ptr(ws), ws_bytes, _status(dev_status),
                                          _stream()))
    return y


def nvfp4_grouped_gemm_workspace_bytes(E: int, M_total: int, N: int, K: int) -> int:
    return int(lib().nvfp4_grouped_gemm_workspace_bytes(E, M_total, N, K))


def nvfp4_gemm_quantize_out(a, sfa, ga, b, sfb, gb, g_out, M: int, N: int, K: int, q_out=None, sf_out=None,
                            dev_status=None, stream=None):
    """y = x . W^T as nvfp4_gemm, emitted as NVFP4 with global scale g_out: returns
    (codes uint8 [M, N/2], tiled scales uint8 [nvfp4_scale_bytes(M, N)])."""
    if stream is not None:
        return _on_stream(stream, nvfp4_gemm_quantize_out, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b, "b"), (sfb, "sfb")):
        _cuda(t, torch.uint8, n)
    for t, n in ((ga, "ga"), (gb, "gb"), (g_out, "g_out")):
        _cuda(t, torch.float32, n)
    if q_out is None:
        q_out = torch.empty((M, N // 2), dtype=torch.uint8, device=a.device)
    if sf_out is None:
        sf_out = torch.empty(nvfp4_scale_bytes(M, N), dtype=torch.uint8, device=a.device)
    _check("nvfp4_gemm_quantize_out",
           lib().nvfp4_gemm_quantize_out(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b), _ptr(sfb), _ptr(gb), _ptr(g_out),
                                         _ptr(q_out), _ptr(sf_out), M, N, K, _status(dev_status), _stream()))
    return q_out, sf_out


def nvfp4_grouped_gemm(a, sfa, ga, b, sfb, gb, expert_offsets, E: int, M_total: int, N: int,
                       K: int, y=None, workspace=None, dev_status=None, stream=None):
    """Per-expert y[rows of e] = x[rows of e] @ W_e^T, rows sorted by expert (bf16 [M_total, N])."""
    if stream is not None:
        return _on_stream(stream, nvfp4_grouped_gemm, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b, "b"), (sfb, "sfb")):
        _cuda(t, torch.uint8, n)
    _cuda(ga, torch.float32, "ga")
    _cuda(gb, torch.float32, "gb")
    _cuda(expert_offsets, torch.int32, "expert_offsets")
    y = torch.empty((M_total, N), dtype=torch.bfloat16, device=a.device) if y is None else y
    ws_bytes = nvfp4_grouped_gemm_workspace_bytes(E, M_total, N, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=a.device)
    _check("nvfp4_grouped_gemm",
           lib().nvfp4_grouped_gemm(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b), _ptr(sfb), _ptr(gb),
                                    _ptr(expert_offsets), E, M_total, N, K, _ptr(y),
                                    _ptr(workspace), workspace.numel(), _status(dev_status),
                                    _stream()))
    return y


def nvfp4_grouped_gemm_gather(a_tok, sfa_tok, ga, b, sfb, gb, expert_offsets, row_token, E: int, T: int,
                              M_total: int, N: int, K: int, y=None, workspace=None, dev_status=None, stream=None):
    """Grouped GEMM over routed rows r (sorted by expert) that read token row row_token[r] of
    the T-row activations a_tok: bf16 [M_total, N] in routed-row order. The default
    workspace has room for the rows to be copied out ahead of the GEMM; one of
    nvfp4_grouped_gemm_workspace_bytes bytes makes the GEMM's load stage gather them."""
    if stream is not None:
        return _on_stream(stream, nvfp4_grouped_gemm_gather, locals())
    for t, n in ((a_tok, "a_tok"), (sfa_tok, "sfa_tok"), (b, "b"), (sfb, "sfb")):
        _cuda(t, torch.uint8, n)
    _cuda(ga, torch.float32, "ga")
    _cuda(gb, torch.float32, "gb")
    _cuda(expert_offsets, torch.int32, "expert_offsets")
    _cuda(row_token, torch.int32, "row_token")
    y = torch.empty((M_total, N), dtype=torch.bfloat16, device=a_tok.device) if y is None else y
    ws_bytes = nvfp4_grouped_gemm_gather_workspace_bytes(E, M_total, N, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=a_tok.device)
    _check("nvfp4_grouped_gemm_gather",
           lib().nvfp4_grouped_gemm_gather(_ptr(a_tok), _ptr(sfa_tok), _ptr(ga), _ptr(b), _ptr(sfb), _ptr(gb),
                                           _ptr(expert_offsets), _ptr(row_token), E, T, M_total, N, K, _ptr(y),
                                           _ptr(workspace), workspace.numel(), _status(dev_status), _stream()))
    return y


def nvfp4_grouped_gemm_gather_workspace_bytes(E: int, M_total: int, N: int, K: int) -> int:
    return int(lib().nvfp4_grouped_gemm_gather_workspace_bytes(E, M_total, N, K))


def nvfp4_grouped_gemm_swiglu(a, sfa, ga, b_gu, sfb_gu, gb, expert_offsets, E: int, M_total: int, N_gu: int,
                              K: int, y=None, workspace=None, dev_status=None, stream=None):
    """Gate/up projection with fused SwiGLU: b_gu interleaves gate and up rows (row 2c gate c,
    2c + 1 up c); returns y[m, c] = silu(gate) * up as bf16 [M_total, N_gu // 2]."""
    if stream is not None:
        return _on_stream(stream, nvfp4_grouped_gemm_swiglu, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b_gu, "b_gu"), (sfb_gu, "sfb_gu")):
        _cuda(t, torch.uint8, n)
    _cuda(ga, torch.float32, "ga")
    _cuda(gb, torch.float32, "gb")
    _cuda(expert_offsets, torch.int32, "expert_offsets")
    y = torch.empty((M_total, N_gu // 2), dtype=torch.bfloat16, device=a.device) if y is None else y
    ws_bytes = nvfp4_grouped_gemm_workspace_bytes(E, M_total, N_gu, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=a.device)
    _check("nvfp4_grouped_gemm_swiglu",
           lib().nvfp4_grouped_gemm_swiglu(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b_gu), _ptr(sfb_gu), _ptr(gb),
                                           _ptr(expert_offsets), E, M_total, N_gu, K, _ptr(y),
                                           _ptr(workspace), workspace.numel(), _status(dev_status),
                                           _stream()))
    return y


NVFP4_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def nvfp4_grouped_gemm_noalloc(a, sfa, ga, b, sfb, gb, expert_offsets, E: int, M_total: int, N: int,
                               K: int, y=None, dev_status=None, stream=None):
    """nvfp4_grouped_gemm without a workspace argument: the library's built-in scratch is used.

    For callers that cannot allocate device memory where they run the MoE layer (runtimes
    with a fixed memory budget and no allocator). Only `y` is allocated here when not given.
    """
    if stream is not None:
        return _on_stream(stream, nvfp4_grouped_gemm_noalloc, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b, "b"), (sfb, "sfb")):
        _cuda(t, torch.uint8, n)
    _cuda(ga, torch.float32, "ga")
    _cuda(gb, torch.float32, "gb")
    _cuda(expert_offsets, torch.int32, "expert_offsets")
    y = torch.empty((M_total, N), dtype=torch.bfloat16, device=a.device) if y is None else y
    _check("nvfp4_grouped_gemm_noalloc",
           lib().nvfp4_grouped_gemm_noalloc(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b), _ptr(sfb), _ptr(gb),
                                            _ptr(expert_offsets), E, M_total, N, K, _ptr(y),
                                            _status(dev_status), _stream()))
    return y


def nvfp4_sparse_meta_bytes(N: int, K: int) -> int:
    return int(lib().nvfp4_sparse_meta_bytes(N, K))


def nvfp4_scale_bytes_b32(rows: int, K: int) -> int:
    return int(lib().nvfp4_scale_bytes_b32(rows, K))


def nvfp4_prune_pairs(w: torch.Tensor, c_out=None, meta_out=None, stream=None):
    """Pair-wise 2:4 pruning + compression of a bf16 weight [N, K]: returns (c bf16 [N, K/2],
    tiled metadata uint8 [nvfp4_sparse_meta_bytes(N, K)])."""
    if stream is not None:
        return _on_stream(stream, nvfp4_prune_pairs, locals())
    _cuda(w, torch.bfloat16, "w")
    N, K = w.shape
    c_out = torch.empty((N, K // 2), dtype=torch.bfloat16, device=w.device) if c_out is None else c_out
    meta_out = (torch.empty(nvfp4_sparse_meta_bytes(N, K), dtype=torch.uint8, device=w.device)
                if meta_out is None else meta_out)
    _check("nvfp4_prune_pairs", lib().nvfp4_prune_pairs(_ptr(w), N, K, _ptr(c_out), _ptr(meta_out),
                                                        _stream()))
    return c_out, meta_out


def nvfp4_quantize_b32(x: torch.Tensor, global_scale: torch.Tensor, q_out=None, sf_out=None, stream=None):
    """bf16 [M, K] -> NVFP4 with 32-element blocks: (q u8 [M, K/2], sf u8 [nvfp4_scale_bytes_b32(M, K)])."""
    if stream is not None:
        return _on_stream(stream, nvfp4_quantize_b32, locals())
    _cuda(x, torch.bfloat16, "x")
    _cuda(global_scale, torch.float32, "global_scale")
    M, K = x.shape
    q_out = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device) if q_out is None else q_out
    sf_out = (torch.empty(nvfp4_scale_bytes_b32(M, K), dtype=torch.uint8, device=x.device)
              if sf_out is None else sf_out)
    _check("nvfp4_quantize_b32", lib().nvfp4_quantize_b32(_ptr(x), M, K, _ptr(global_scale), _ptr(q_out),
                                                          _ptr(sf_out), _stream()))
    return q_out, sf_out


def nvfp4_grouped_gemm_swiglu_quantize_out(a, sfa, ga, b_gu, sfb_gu, gb, expert_offsets, E: int, M_total: int,
                                           N_gu: int, K: int, g_out, q_out=None, sf_out=None, workspace=None,
                                           dev_status=None, stream=None):
    """Gate/up projection with SwiGLU emitting NVFP4 with the global scale g_out: returns
    (codes u8 [M_total, N_gu // 4], tiled scales u8 [nvfp4_scale_bytes(M_total, N_gu // 2)])."""
    if stream is not None:
        return _on_stream(stream, nvfp4_grouped_gemm_swiglu_quantize_out, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b_gu, "b_gu"), (sfb_gu, "sfb_gu")):
        _cuda(t, torch.uint8, n)
    for t, n in ((ga, "ga"), (gb, "gb"), (g_out, "g_out")):
        _cuda(t, torch.float32, n)
    dev = a.device
    q_out = torch.empty((M_total, N_gu // 4), dtype=torch.uint8, device=dev) if q_out is None else q_out
    sf_out = (torch.empty(nvfp4_scale_bytes(M_total, N_gu // 2), dtype=torch.uint8, device=dev)
              if sf_out is None else sf_out)
    ws_bytes = int(lib().nvfp4_grouped_gemm_workspace_bytes(E, M_total, N_gu, K))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    _check("nvfp4_grouped_gemm_swiglu_quantize_out",
           lib().nvfp4_grouped_gemm_swiglu_quantize_out(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b_gu), _ptr(sfb_gu),
                                                        _ptr(gb), _ptr(expert_offsets), E, M_total, N_gu, K,
                                                        _ptr(g_out), _ptr(q_out), _ptr(sf_out), _ptr(workspace),
                                                        workspace.numel(), _status(dev_status), _stream()))
    return q_out, sf_out


def nvfp4_gemm_batched(problems, M: int, dev_status=None, stream=None):
    """Several decode-M GEMMs in one launch. problems: sequence of (a, sfa, ga, b, sfb, gb, y)
    tuples of CUDA tensors (y bf16 [M, N], preallocated); N and K come from b and a."""
    if stream is not None:
        return _on_stream(stream, nvfp4_gemm_batched, locals())
    arr = (GemmProblem * max(1, len(problems)))()
    for i, (a, sfa, ga, b, sfb, gb, y) in enumerate(problems):
        for t, n in ((a, "a"), (sfa, "sfa"), (b, "b"), (sfb, "sfb")):
            _cuda(t, torch.uint8, n)
        _cuda(ga, torch.float32, "ga")
        _cuda(gb, torch.float32, "gb")
        _cuda(y, torch.bfloat16, "y")
        arr[i] = GemmProblem(a.data_ptr(), sfa.data_ptr(), ga.data_ptr(), b.data_ptr(), sfb.data_ptr(),
                             gb.data_ptr(), y.data_ptr(), b.shape[0], 2 * b.shape[1])
    _check("nvfp4_gemm_batched", lib().nvfp4_gemm_batched(ctypes.cast(arr, ctypes.c_void_p), len(problems), M,
                                                          _status(dev_status), _stream()))


def nvfp4_sparse_gemm(a, sfa, ga, b_c, sfb_c, meta, gb, M: int, N: int, K: int, y=None, dev_status=None,
                      stream=None):
    """y = x @ W^T, W pair-wise 2:4 sparse (compressed codes b_c [N, K/4], scales sfb_c, tiled meta),
    x in 32-element blocks; bf16 [M, N]."""
    if stream is not None:
        return _on_stream(stream, nvfp4_sparse_gemm, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b_c, "b_c"), (sfb_c, "sfb_c"), (meta, "meta")):
        _cuda(t, torch.uint8, n)
    _cuda(ga, torch.float32, "ga")
    _cuda(gb, torch.float32, "gb")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=a.device) if y is None else y
    _check("nvfp4_sparse_gemm", lib().nvfp4_sparse_gemm(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b_c), _ptr(sfb_c),
                                                        _ptr(meta), _ptr(gb), _ptr(y), M, N, K, _status(dev_status),
                                                        _stream()))
    return y


def nvfp4_grouped_sparse_gemm(a, sfa, ga, b_c, sfb_c, meta, gb, expert_offsets, E: int, M_total: int, N: int,
                              K: int, y=None, workspace=None, dev_status=None, stream=None):
    """Grouped form of nvfp4_sparse_gemm over pair-wise 2:4 sparse experts; bf16 [M_total, N]."""
    if stream is not None:
        return _on_stream(stream, nvfp4_grouped_sparse_gemm, locals())
    for t, n in ((a, "a"), (sfa, "sfa"), (b_c, "b_c"), (sfb_c, "sfb_c"), (meta, "meta")):
        _cuda(t, torch.uint8, n)
    _cuda(ga, torch.float32, "ga")
    _cuda(gb, torch.float32, "gb")
    _cuda(expert_offsets, torch.int32, "expert_offsets")
    y = torch.empty((M_total, N), dtype=torch.bfloat16, device=a.device) if y is None else y
    if workspace is None:
        workspace = torch.empty(max(1, nvfp4_grouped_gemm_workspace_bytes(E, M_total, N, K)), dtype=torch.uint8,
                                device=a.device)
    _check("nvfp4_grouped_sparse_gemm",
           lib().nvfp4_grouped_sparse_gemm(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b_c), _ptr(sfb_c), _ptr(meta),
                                           _ptr(gb), _ptr(expert_offsets), E, M_total, N, K, _ptr(y),
                                           _ptr(workspace), workspace.numel(), _status(dev_status), _stream()))
    return y


NVFP4_BF16 = 0
NVFP4_F32 = 1
NVFP4_MOE_MAX_EXPERTS = 1024
NVFP4_MOE_MAX_TOPK = 32
_FLOAT_TYPES = {torch.bfloat16: NVFP4_BF16, torch.float32: NVFP4_F32}


_FP8_TYPES = (torch.float8_e4m3fn, torch.uint8)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U8 = (torch.uint8,)
_BF16 = (torch.bfloat16,)


def _fits(have, shape):
    """Whether a contiguous tensor of sizes `have` holds one of `shape` at its start: as many elements, and, unless
    it is a flat buffer, rows of the same length. Dimensions may be merged or split ([tokens, heads, size] for
    [tokens, K]) and there may be more rows."""
    if math.prod(have) < math.prod(shape):
        return False
    runs = [1] + [math.prod(have[-i:]) for i in range(1, len(have) + 1)]  # elements of the inner slices
    inner = min(len(have), len(shape))
    return all(math.prod(shape[-i:]) in runs for i in range(1, inner))


def _operand(t, types, shape, name):
    """t's address; t must be a contiguous CUDA tensor of one of `types` whose memory starts with a tensor of
    `shape` (see _fits)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in types and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous CUDA tensor of {' or '.join(map(str, types))}")
    if t.shape != shape and not _fits(t.shape, shape):
        raise TypeError(f"{name} has shape {tuple(t.shape)}, needs {shape}")
    return t.data_ptr()


@functools.lru_cache(maxsize=128)
def _routing_layout(T, E, k):
    """The one description of a MoeRouting's buffer: the fields as {name: (first word, shape, strides, fp32)} in
    the order in which they lie there, which is MoeRouting._fields and the order of nvfp4_moe_route's arguments;
    the byte offsets of all of them and of the workspace behind them (16-byte aligned); the words up to it."""
    n = max(T * k, 0)  # (a negative k is the library's to refuse)
    per = ((T, k), (k, 1), n)

    def row(size):
        return (size,), (1,), size

    fields, at = {}, 0
    for name, (size, strides, words), fp32 in (
            ("topk_idx", per, False), ("topk_w", per, True), ("slot_row", per, False), ("counts", row(E), False),
            ("expert_offsets", row(E + 1), False), ("row_token", row(n), False), ("mean_prob", row(E), True),
            ("balance_loss", row(1), True), ("routed_tokens", row(1), False)):
        fields[name] = (at, size, strides, fp32)
        at += words
    words = (at + 3) // 4 * 4
    return fields, tuple(4 * f[0] for f in fields.values()) + (4 * words,), words


class MoeRouting:
    """What nvfp4_moe_route returns (T tokens, k slots each, E experts): tensors that share one
    allocation, as attributes made when they are first asked for (a call's host time is mostly
    that of making tensors).

    topk_idx        int32 [T, k]: selected experts, -1 in empty slots
    topk_w          fp32 [T, k]: their weights
    slot_row        int32 [T, k]: routed row of each slot, -1 in empty slots
    row_token       int32 [T * k]: token of each routed row, -1 past the last
    counts          int32 [E]: rows per expert
    expert_offsets  int32 [E + 1]: as the grouped GEMMs read them
    mean_prob       fp32 [E]: mean probability over the routed tokens
    balance_loss    fp32 [1]
    routed_tokens   int32 [1]

    It also keeps what the call was given and its gradient depends on: renormalize and valid (the tensor
    itself, which has to hold the same at the backward call).
    """
    _fields = ("topk_idx", "topk_w", "slot_row", "counts", "expert_offsets", "row_token", "mean_prob", "balance_loss",
               "routed_tokens")

    def __init__(self, T, E, k, renormalize, valid, device, workspace_words):
        self.T, self.E, self.k, self.renormalize, self.valid = T, E, k, renormalize, valid
        self._all = self._float = None
        self._layout = layout = _routing_layout(T, E, k)
        self._buf = torch.empty(layout[2] + workspace_words, dtype=torch.int32, device=device)

    def __getstate__(self):  # for copies: the views are made anew
        return {f: self.__dict__[f] for f in ("T", "E", "k", "renormalize", "valid", "_layout", "_buf")} | {
            "_all": None, "_float": None}

    def _addresses(self):
        """Of the fields, in their order, and of the workspace behind them."""
        base = self._buf.data_ptr()
        return [base + at for at in self._layout[1]]

    def _floats(self):
        if self._float is None:
            self._float = self._buf.view(torch.float32)
        return self._float

    def __getattr__(self, name):  # only for what is not there yet
        if name not in MoeRouting._fields:
            raise AttributeError(name)
        at, size, strides, fp32 = self._layout[0][name]
        t = self.__dict__[name] = (self._floats() if fp32 else self._buf).as_strided(size, strides, at)
        return t

    def _asdict(self):
        made = self._all
        if made is None:
            views, floats, have = self._buf.as_strided, self._floats().as_strided, self.__dict__
            made = self._all = {}
            for name, (at, size, strides, fp32) in self._layout[0].items():
                t = have.get(name)  # those handed out before stay
                if t is None:
                    t = have[name] = floats(size, strides, at) if fp32 else views(size, strides, at)
                made[name] = t
        return dict(made)

    def __iter__(self):
        return iter(self._asdict().values())


def _route_inputs(logits, valid):
    """T and E of the logits, and the address of valid."""
    if not (isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dtype in _FLOAT_TYPES
            and logits.is_contiguous() and logits.dim() == 2):
        raise TypeError("logits must be a contiguous CUDA tensor [T, E] of torch.bfloat16 or torch.float32")
    if valid is not None and not (isinstance(valid, torch.Tensor) and valid.is_cuda and valid.is_contiguous()
                                  and valid.dtype in (torch.bool, torch.uint8) and valid.numel() == logits.shape[0]):
        raise TypeError("valid must be a contiguous CUDA tensor [T] of torch.bool or torch.uint8")
    return *logits.shape, None if valid is None else valid.data_ptr()


def nvfp4_moe_route_workspace_bytes(T: int, E: int) -> int:
    return int(lib().nvfp4_moe_route_workspace_bytes(T, E))


_route_workspace_bytes = functools.lru_cache(maxsize=128)(nvfp4_moe_route_workspace_bytes)


def nvfp4_moe_route(logits: torch.Tensor, k: int, renormalize: bool = False, valid=None, workspace=None,
                    stream=None) -> MoeRouting:
    """Softmax router: top-k experts and weights of each token, per-expert counts and offsets, the
    expert-sorted row lists that the grouped GEMMs read, and the load-balance loss."""
    if stream is not None:
        return _on_stream(stream, nvfp4_moe_route, locals())
    T, E, on = _route_inputs(logits, valid)
    ws_bytes = _route_workspace_bytes(T, E)
    renormalize = bool(renormalize)
    r = MoeRouting(T, E, k, renormalize, valid, logits.device, ws_bytes // 4 if workspace is None else 0)
    *fields, ws = r._addresses()
    if workspace is not None:
        ws, ws_bytes = _operand(workspace, _U8, (0,), "workspace"), workspace.numel()
    _check("nvfp4_moe_route",
           lib().nvfp4_moe_route(logits.data_ptr(), _FLOAT_TYPES[logits.dtype], on, T, E, k, renormalize, *fields,
                                 ws, ws_bytes, _stream()))
    return r


def nvfp4_moe_route_backward(logits: torch.Tensor, routing: MoeRouting, d_w=None, d_loss=None,
                             renormalize=None, valid=None, d_logits=None, stream=None) -> torch.Tensor:
    """Gradient of nvfp4_moe_route's logits from the gradients of the weights topk_w (d_w, fp32 [T, k])
    and of the balance loss (d_loss, fp32 [1]). renormalize and valid are those of the routing; given
    here, they have to agree with it."""
    if stream is not None:
        return _on_stream(stream, nvfp4_moe_route_backward, locals())
    if valid is None:
        valid = routing.valid
    elif routing.valid is None:
        raise TypeError("the routing was made without valid")
    T, E, on = _route_inputs(logits, valid)
    k = routing.k
    if (routing.T, routing.E) != (T, E):
        raise TypeError(f"routing is of {routing.T} tokens and {routing.E} experts, logits of {T} and {E}")
    if renormalize is not None and bool(renormalize) != routing.renormalize:
        raise TypeError(f"the routing was made with renormalize={routing.renormalize}")
    for t, shape, n in ((d_w, (T, k), "d_w"), (d_loss, (1,), "d_loss")):
        if t is not None:
            _cuda(t, torch.float32, n)
            if tuple(t.shape) != shape:
                raise TypeError(f"{n} must have shape {shape}")
    d_logits = torch.empty_like(logits) if d_logits is None else d_logits
    topk_idx, topk_w, _, counts, _, _, _, _, routed_tokens, _ = routing._addresses()
    _check("nvfp4_moe_route_backward",
           lib().nvfp4_moe_route_backward(logits.data_ptr(), _FLOAT_TYPES[logits.dtype], on, T, E, k,
                                          routing.renormalize, topk_idx, topk_w, counts, routed_tokens, _ptr(d_w),
                                          _ptr(d_loss), _operand(d_logits, (logits.dtype,), (T, E), "d_logits"), _stream()))
    return d_logits


def _blocks(n):
    return (n + 127) // 128


def nvfp4_fp8_quantize(x: torch.Tensor, block_rows: int = 1, row_token=None, transposed: bool = False, stream=None):
    """bf16 [M, K] -> (codes float8_e4m3fn [M, K], scales fp32), one scale per 1 x 128 block along K
    (scales [K/128, M]) or, with block_rows=128, per 128 x 128 block (scales [M/128, K/128]; sizes
    rounded up). row_token (int32): quantise the rows x[row_token]. transposed: also return the
    codes [K, M rounded up to 16] and scales of the transpose, blocks along M."""
    if stream is not None:
        return _on_stream(stream, nvfp4_fp8_quantize, locals())
    _cuda(x, torch.bfloat16, "x")
    if x.dim() != 2:
        raise TypeError("x must be [M, K]")
    M_x, K = x.shape
    M, rows, transpose = M_x, None, (None, None)
    if row_token is not None:
        _cuda(row_token, torch.int32, "row_token")
        M, rows = row_token.numel(), row_token.data_ptr()
    dev = x.device
    square = block_rows == 128
    q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
    s = torch.empty((_blocks(M), _blocks(K)) if square else (_blocks(K), M), dtype=torch.float32, device=dev)
    if transposed:
        qt = torch.empty((K, (M + 15) // 16 * 16), dtype=torch.float8_e4m3fn, device=dev)
        st = torch.empty((_blocks(K), _blocks(M)) if square else (_blocks(M), K), dtype=torch.float32, device=dev)
        transpose = qt.data_ptr(), st.data_ptr()
    _check("nvfp4_fp8_quantize",
           lib().nvfp4_fp8_quantize(x.data_ptr(), M_x, K, block_rows, rows, M, q.data_ptr(), s.data_ptr(), *transpose,
                                    _stream()))
    return (q, s, qt, st) if transposed else (q, s)


def nvfp4_fp8_gemm(a, sa, b, sb, M: int, N: int, K: int, b_block_rows: int = 128, out_dtype=torch.bfloat16, y=None,
                   dev_status=None, stream=None):
    """y = a b^T [M, N] in bf16 or fp32 from E4M3 codes a [M, K], b [N, K] and their block scales
    (see nvfp4_fp8_quantize; b_block_rows: rows of b that share a scale, 128 or 1)."""
    if stream is not None:
        return _on_stream(stream, nvfp4_fp8_gemm, locals())
    y_type = _FLOAT_TYPES.get(out_dtype)
    if y_type is None:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    kb = _blocks(K)
    try:
        pa = _operand(a, _FP8_TYPES, (M, K), "a")
        args = (pa, _operand(sa, _F32, (kb, M), "sa"), _operand(b, _FP8_TYPES, (N, K), "b"),
                _operand(sb, _F32, (kb, N) if b_block_rows == 1 else (_blocks(N), kb), "sb"), b_block_rows)
        if y is None:
            y = torch.empty((M, N), dtype=out_dtype, device=a.device)
            py = y.data_ptr()
        else:
            py = _operand(y, (out_dtype,), (M, N), "y")
    except TypeError:  # sizes that the library refuses are its error
        _check("nvfp4_fp8_gemm", lib().nvfp4_fp8_gemm(None, None, None, None, b_block_rows, None, y_type, min(M, 0), N, K,
                                                      None, None))
        raise
    _check("nvfp4_fp8_gemm", lib().nvfp4_fp8_gemm(*args, py, y_type, M, N, K, _status(dev_status), _stream()))
    return y


def nvfp4_fp8_grouped_gemm_workspace_bytes(E: int, M_total: int, N: int, K: int) -> int:
    return int(lib().nvfp4_fp8_grouped_gemm_workspace_bytes(E, M_total, N, K))


_fp8_grouped_workspace_bytes = functools.lru_cache(maxsize=128)(nvfp4_fp8_grouped_gemm_workspace_bytes)


def nvfp4_fp8_grouped_gemm(a, sa, b, sb, expert_offsets, E: int, M_total: int, N: int, K: int, y=None,
                           workspace=None, dev_status=None, stream=None):
    """Per-expert y[rows of e] = a[rows of e] b_e^T (bf16 [M_total, N]) from E4M3 codes a [M_total, K],
    b [E, N, K] and their block scales; rows sorted by expert, rows past expert_offsets[E] untouched."""
    if stream is not None:
        return _on_stream(stream, nvfp4_fp8_grouped_gemm, locals())
    kb = _blocks(K)
    try:
        pa = _operand(a, _FP8_TYPES, (M_total, K), "a")
        args = (pa, _operand(sa, _F32, (kb, M_total), "sa"), _operand(b, _FP8_TYPES, (E, N, K), "b"),
                _operand(sb, _F32, (E, _blocks(N), kb), "sb"), _operand(expert_offsets, _I32, (E + 1,), "expert_offsets"),
                E, M_total, N, K)
        if y is None:
            y = torch.empty((M_total, N), dtype=torch.bfloat16, device=a.device)
            py = y.data_ptr()
        else:
            py = _operand(y, _BF16, (M_total, N), "y")
    except TypeError:  # sizes that the library refuses are its error
        _check("nvfp4_fp8_grouped_gemm",
               lib().nvfp4_fp8_grouped_gemm(None, None, None, None, None, E, min(M_total, 0), N, K, None, None, 0, None, None))
        raise
    if workspace is None:
        ws_bytes = max(1, _fp8_grouped_workspace_bytes(E, M_total, N, K))
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=a.device)
        pws = workspace.data_ptr()
    else:
        pws, ws_bytes = _operand(workspace, _U8, (0,), "workspace"), workspace.numel()
    _check("nvfp4_fp8_grouped_gemm",
           lib().nvfp4_fp8_grouped_gemm(*args, py, pws, ws_bytes, _status(dev_status), _stream()))
    return y


NVFP4_F16 = 2
NVFP4_SILU = 0
NVFP4_GELU_TANH = 1
_HALF_TYPES = {torch.bfloat16: NVFP4_BF16, torch.float16: NVFP4_F16}
_ACTIVATIONS = {"silu": NVFP4_SILU, "gelu_tanh": NVFP4_GELU_TANH}


def nvfp4_gated_ffn_workspace_bytes(M: int, I: int, K: int) -> int:
    return int(lib().nvfp4_gated_ffn_workspace_bytes(M, I, K))


def nvfp4_gated_ffn_backward_workspace_bytes(M: int, I: int, K: int) -> int:
    return int(lib().nvfp4_gated_ffn_backward_workspace_bytes(M, I, K))


_ffn_workspace_bytes = functools.lru_cache(maxsize=128)(nvfp4_gated_ffn_workspace_bytes)
_ffn_backward_workspace_bytes = functools.lru_cache(maxsize=128)(nvfp4_gated_ffn_backward_workspace_bytes)


def _rows(t, dtype, shape, name):
    """Address and row stride of a matrix of `shape` on the current device, whose rows may lie apart."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype):
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.shape != shape:
        raise TypeError(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
    if t.get_device() != torch._C._cuda_getDevice():
        raise TypeError(f"{name} is on {t.device}, not on the current device")
    ld, step = t.stride()
    if shape[0] <= 1 or 0 in shape:  # no second row: the stride says nothing
        ld = shape[1]
    if step != 1 and shape[1] != 1 or ld < shape[1]:
        raise TypeError(f"{name} must have contiguous rows, one behind the other")
    return t.data_ptr(), ld


def _here(*tensors):
    """Refuses tensors that lie on another device than the current one."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise TypeError(f"a tensor is on {t.device}, not on the current device")


def _ffn_inputs(x, w_gate, w_up, activation):
    """M, I, K, the codes of the type and of the activation."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in _HALF_TYPES and x.dim() == 2):
        raise TypeError("x must be a CUDA tensor [M, K] of torch.bfloat16 or torch.float16")
    if not (isinstance(w_gate, torch.Tensor) and w_gate.dim() == 2):
        raise TypeError("w_gate must be a CUDA tensor [I, K]")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}")
    return x.shape[0], w_gate.shape[0], x.shape[1], _HALF_TYPES[x.dtype], act


def nvfp4_gated_ffn(x, w_gate, w_up, activation="silu", save=False, h=None, workspace=None, dev_status=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T), bf16 or fp16: x [M, K], w_gate and w_up [I, K], h [M, I]; activation
    "silu" or "gelu_tanh". With save, returns (h, gate, up): the two products in fp32, for nvfp4_gated_ffn_backward. The rows of
    x, the weights and h may lie apart (views of wider tensors); their strides, I and K are multiples of 8."""
    if stream is not None:
        return _on_stream(stream, nvfp4_gated_ffn, locals())
    M, I, K, kind, act = _ffn_inputs(x, w_gate, w_up, activation)
    dtype, dev = x.dtype, x.device
    args = _rows(x, dtype, (M, K), "x") + _rows(w_gate, dtype, (I, K), "w_gate") + _rows(w_up, dtype, (I, K), "w_up")
    h = torch.empty((M, I), dtype=dtype, device=dev) if h is None else h
    ph, ldh = _rows(h, dtype, (M, I), "h")
    gate = up = pg = pu = None
    if save:
        gate, up = torch.empty((M, I), dtype=torch.float32, device=dev), torch.empty((M, I), dtype=torch.float32, device=dev)
        pg, pu = gate.data_ptr(), up.data_ptr()
    ws_bytes, pws = _ffn_workspace_bytes(M, I, K), None
    _here(workspace, dev_status)
    if workspace is not None:
        pws, ws_bytes = _operand(workspace, _U8, (0,), "workspace"), workspace.numel()
    elif ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        pws = workspace.data_ptr()
    _check("nvfp4_gated_ffn", lib().nvfp4_gated_ffn(*args, kind, act, ph, ldh, pg, pu, M, I, K, pws, ws_bytes,
                                                    _status(dev_status), _stream()))
    return (h, gate, up) if save else h


def nvfp4_gated_ffn_backward(x, w_gate, w_up, gate, up, dh, activation="silu", need=(True, True, True), dx=None,
                             dw_gate=None, dw_up=None, workspace=None, dev_status=None, stream=None):
    """(dx, dw_gate, dw_up) of nvfp4_gated_ffn from its gate and up and the gradient dh [M, I] of h, in the operands'
    type; `need` says which are wanted (None for the others). The gradients are contiguous."""
    if stream is not None:
        return _on_stream(stream, nvfp4_gated_ffn_backward, locals())
    M, I, K, kind, act = _ffn_inputs(x, w_gate, w_up, activation)
    dtype, dev = x.dtype, x.device
    args = _rows(x, dtype, (M, K), "x") + _rows(w_gate, dtype, (I, K), "w_gate") + _rows(w_up, dtype, (I, K), "w_up")
    for t, n in ((gate, "gate"), (up, "up")):
        if _rows(t, torch.float32, (M, I), n)[1] != I:
            raise TypeError(f"{n} must be contiguous")
        args += (t.data_ptr(),)
    args += _rows(dh, dtype, (M, I), "dh")
    if len(need) != 3:
        raise ValueError("need says for dx, dw_gate and dw_up whether they are wanted")
    _here(workspace, dev_status)
    outs, ptrs = [], []
    for t, wanted, shape, n in zip((dx, dw_gate, dw_up), need, ((M, K), (I, K), (I, K)), ("dx", "dw_gate", "dw_up")):
        if wanted and t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        elif wanted and _rows(t, dtype, shape, n)[1] != K:
            raise TypeError(f"{n} must be contiguous")
        outs.append(t if wanted else None)
        ptrs.append(t.data_ptr() if wanted else None)
    if workspace is None:
        ws_bytes = _ffn_backward_workspace_bytes(M, I, K)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        pws = workspace.data_ptr()
    else:
        pws, ws_bytes = _operand(workspace, _U8, (0,), "workspace"), workspace.numel()
    _check("nvfp4_gated_ffn_backward",
           lib().nvfp4_gated_ffn_backward(*args, kind, act, *ptrs, M, I, K, pws, ws_bytes, _status(dev_status), _stream()))
    return tuple(outs)


def nvfp4_int8_quantize(x: torch.Tensor, stream=None):
    """bf16 or fp16 [M, K] -> (codes int8 [M, K], scales fp32 [M]): the largest magnitude of a row becomes 127. The
    rows of x may lie apart. Weights [N, K] are quantised for each output channel by the same call."""
    if stream is not None:
        return _on_stream(stream, nvfp4_int8_quantize, locals())
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in _HALF_TYPES and x.dim() == 2):
        raise TypeError("x must be a CUDA tensor [M, K] of torch.bfloat16 or torch.float16")
    M, K = x.shape
    px, ldx = _rows(x, x.dtype, (M, K), "x")
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s = torch.empty(M, dtype=torch.float32, device=x.device)
    _check("nvfp4_int8_quantize",
           lib().nvfp4_int8_quantize(px, ldx, _HALF_TYPES[x.dtype], M, K, q.data_ptr(), s.data_ptr(), _stream()))
    return q, s


_I8 = (torch.int8,)
_OUT_TYPES = {torch.bfloat16: NVFP4_BF16, torch.float32: NVFP4_F32, torch.float16: NVFP4_F16}


def nvfp4_int8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().nvfp4_int8_gemm_workspace_bytes(M, N, K))


_int8_workspace_bytes = functools.lru_cache(maxsize=128)(nvfp4_int8_gemm_workspace_bytes)


def nvfp4_int8_gemm(a, sa, b, sb, M: int, N: int, K: int, out_dtype=torch.bfloat16, y=None, workspace=None, dev_status=None,
                    stream=None):
    """y = sa[m] sb[n] (a b^T) [M, N] in bf16, fp16 or fp32 from int8 codes a [M, K], b [N, K] and their row scales
    (see nvfp4_int8_quantize); the integer sums are exact."""
    if stream is not None:
        return _on_stream(stream, nvfp4_int8_gemm, locals())
    y_type = _OUT_TYPES.get(out_dtype)
    if y_type is None:
        raise TypeError("out_dtype must be torch.bfloat16, torch.float16 or torch.float32")
    try:
        pa = _operand(a, _I8, (M, K), "a")
        args = (pa, _operand(sa, _F32, (M,), "sa"), _operand(b, _I8, (N, K), "b"), _operand(sb, _F32, (N,), "sb"))
        if y is None:
            y = torch.empty((M, N), dtype=out_dtype, device=a.device)
            py = y.data_ptr()
        else:
            py = _operand(y, (out_dtype,), (M, N), "y")
    except TypeError:  # sizes that the library refuses are its error
        _check("nvfp4_int8_gemm", lib().nvfp4_int8_gemm(None, None, None, None, None, y_type, min(M, 0), N, K, None, 0, None, None))
        raise
    _here(a, sa, b, sb, y, workspace, dev_status)
    ws_bytes, pws = _int8_workspace_bytes(M, N, K), None
    if workspace is not None:
        pws, ws_bytes = _operand(workspace, _U8, (0,), "workspace"), workspace.numel()
    elif ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=a.device)
        pws = workspace.data_ptr()
    _check("nvfp4_int8_gemm",
           lib().nvfp4_int8_gemm(*args, py, y_type, M, N, K, pws, ws_bytes, _status(dev_status), _stream()))
    return y


_GRAD_TYPES = {torch.bfloat16: NVFP4_BF16, torch.float32: NVFP4_F32, torch.float16: NVFP4_F16}


def nvfp4_grad_clip_workspace_bytes(count: int) -> int:
    return int(lib().nvfp4_grad_clip_workspace_bytes(count))


_clip_workspace_bytes = functools.lru_cache(maxsize=128)(nvfp4_grad_clip_workspace_bytes)


@functools.lru_cache(maxsize=128)
def _list_types(n):  # of the host arrays of n gradients: making the types takes longer than filling them
    return _vp * n, _i64 * n, _i32 * n


def nvfp4_grad_clip(grads, max_norm=math.inf, out=None, norm=None, workspace=None, stream=None) -> torch.Tensor:
    """The norm over all values of `grads` (contiguous CUDA tensors, bf16, fp16 or fp32, mixed as they come), fp32 [1];
    the gradients are multiplied by min(1, max_norm / (norm + 1e-6)), in place or into the tensors `out` of the same
    types and shapes. Without max_norm only the norm is computed. No two results may share memory."""
    if stream is not None:
        return _on_stream(stream, nvfp4_grad_clip, locals())
    grads = list(grads)
    n = len(grads)
    dev, (pointers, counts, kinds) = grads[0].device if n else "cuda", _list_types(n)
    # list by list: a list's check costs half of one tensor by tensor, and lists may be long
    here, types = [torch._C._cuda_getDevice()] * n, [t.dtype for t in grads]
    if [t.get_device() for t in grads] != here or not _GRAD_TYPES.keys() >= set(types) or not all([t.is_contiguous() for t in grads]):
        raise TypeError("grads must be contiguous tensors of torch.bfloat16, float16 or float32 on the current CUDA device")
    to = None
    if out is not None:
        out = list(out)
        if ([o.dtype for o in out] != types or [o.get_device() for o in out] != here or [o.shape for o in out] != [t.shape for t in grads]
                or not all([o.is_contiguous() for o in out])):
            raise TypeError("out must hold contiguous tensors of the types and shapes of grads, on the same device")
        to = pointers(*[o.data_ptr() for o in out])
    _here(norm, workspace)
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(_clip_workspace_bytes(n), dtype=torch.uint8, device=dev)
    _check("nvfp4_grad_clip",
           lib().nvfp4_grad_clip(pointers(*[t.data_ptr() for t in grads]), to, counts(*[t.numel() for t in grads]),
                                 kinds(*[_GRAD_TYPES[t] for t in types]), n, max_norm, _operand(norm, _F32, (1,), "norm"),
                                 _operand(workspace, _U8, (0,), "workspace"), workspace.numel(), _stream()))
    return norm


def nvfp4_encode_e2m1(v: torch.Tensor, stream=None) -> torch.Tensor:
    if stream is not None:
        return _on_stream(stream, nvfp4_encode_e2m1, locals())
    _cuda(v, torch.float32, "v")
    out = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check("nvfp4_encode_e2m1", lib().nvfp4_encode_e2m1(_ptr(v), v.numel(), _ptr(out), _stream()))
    return out


def nvfp4_encode_e4m3(v: torch.Tensor, stream=None) -> torch.Tensor:
    if stream is not None:
        return _on_stream(stream, nvfp4_encode_e4m3, locals())
    _cuda(v, torch.float32, "v")
    out = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check("nvfp4_encode_e4m3", lib().nvfp4_encode_e4m3(_ptr(v), v.numel(), _ptr(out), _stream()))
    return out
