"""ctypes binding of libnvfp4.so (include/nvfp4.h): argument marshalling only.

Every function here has the name of the C entry point it calls and does
nothing but turn PyTorch tensors into pointers, sizes and the current CUDA
stream.  All arithmetic runs in the library's CUDA kernels.  If the library is
missing or fails to load, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import struct
import threading
from dataclasses import dataclass

import torch

from . import build as _build

NVFP4_OK = 0
NVFP4_ERR_INVALID_ARG = 1
NVFP4_ERR_UNSUPPORTED_SHAPE = 2
NVFP4_ERR_WORKSPACE = 3
NVFP4_ERR_CUDA = 4
NVFP4_ERR_DEVICE_TIMEOUT = 5
NVFP4_ERR_DEVICE_INDEX = 6

NVFP4_STATUS_WORD_OFFSET = 128

NVFP4_OP_QUANTIZE = 0
NVFP4_OP_GEMV_SKINNY = 1
NVFP4_OP_GATEUP_SWIGLU = 2
NVFP4_OP_GEMM_PREFILL = 3
NVFP4_OP_FP6_GEMM = 4
NVFP4_OP_FP6_GATEUP_SWIGLU = 5
NVFP4_OP_KV_APPEND = 6

NVFP4_OUT_F32 = 0
NVFP4_OUT_BF16 = 1

NVFP4_ACT_NONE = 0
NVFP4_ACT_SILU = 1
NVFP4_ACT_GELU = 2
NVFP4_ACT_GELU_TANH = 3
NVFP4_ACT_RELU = 4
NVFP4_ACT_RELU2 = 5

NVFP4_KV_E4M3 = 0
NVFP4_KV_NVFP4 = 1

_lock = threading.Lock()
_lib = None


class SkinnyJobC(ctypes.Structure):
    """nvfp4_skinny_job of include/nvfp4.h."""
    _fields_ = [("x", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("input", ctypes.c_int32),
                ("n_weights", ctypes.c_int32), ("codes", ctypes.c_void_p * 2), ("scales", ctypes.c_void_p * 2),
                ("tensor_scale", ctypes.c_void_p * 2), ("M", ctypes.c_int64), ("K", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class KVCacheC(ctypes.Structure):
    """nvfp4_kv_cache of include/nvfp4.h."""
    _fields_ = [("pool", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class PagedAttentionArgsC(ctypes.Structure):
    """nvfp4_paged_attention_args of include/nvfp4.h."""
    _fields_ = [("cache", KVCacheC), ("q", ctypes.c_void_p), ("q_ld", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_ld", ctypes.c_int64), ("block_table", ctypes.c_void_p), ("table_width", ctypes.c_int64),
                ("kv_lens", ctypes.c_void_p), ("q_offsets", ctypes.c_void_p), ("tree", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int64), ("total_q", ctypes.c_int64), ("max_q_len", ctypes.c_int64),
                ("window", ctypes.c_int64), ("n_q_heads", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", ctypes.c_float)]


class RopePairC(ctypes.Structure):
    """nvfp4_rope_pair of include/nvfp4.h."""
    _fields_ = [("turn", ctypes.c_uint64), ("axis", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class RopeArgsC(ctypes.Structure):
    """nvfp4_rope_args of include/nvfp4.h."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_ld", ctypes.c_int64), ("k_ld", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("q_out_ld", ctypes.c_int64),
                ("k_out_ld", ctypes.c_int64), ("positions", ctypes.c_void_p), ("positions_ld", ctypes.c_int64),
                ("pairs", ctypes.c_void_p), ("n_tokens", ctypes.c_int64), ("n_axes", ctypes.c_int32),
                ("n_pairs", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_k_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("adjacent", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class EpilogueC(ctypes.Structure):
    """nvfp4_epilogue of include/nvfp4.h."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("residual_ld", ctypes.c_int64),
                ("bias_dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class PromptAttentionArgsC(ctypes.Structure):
    """nvfp4_prompt_attention_args of include/nvfp4.h."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_ld", ctypes.c_int64),
                ("k_ld", ctypes.c_int64), ("v_ld", ctypes.c_int64), ("out", ctypes.c_void_p), ("out_ld", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("n_seqs", ctypes.c_int64), ("total", ctypes.c_int64),
                ("window", ctypes.c_int64), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {nvfp4_status_string(status)} (status {status})")


def library_path() -> str:
    return _build.LIB


def load_library():
    """Load libnvfp4.so (built by gemm_nvfp4_gb300.build / __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"libnvfp4.so not found at {path}: build it with `python -m gemm_nvfp4_gb300.build` "
                "(the NVFP4 path has no CPU fallback)")
        lib = ctypes.CDLL(path)
        P, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        lib.nvfp4_status_string.restype = ctypes.c_char_p
        lib.nvfp4_status_string.argtypes = [i32]
        lib.nvfp4_version.restype = i32
        lib.nvfp4_version.argtypes = []
        lib.nvfp4_workspace_bytes.restype = sz
        lib.nvfp4_workspace_bytes.argtypes = [i32, i64, i64, i64]
        lib.nvfp4_quantize.restype = i32
        lib.nvfp4_quantize.argtypes = [P, i64, i64, P, P, P, P, sz, P]
        lib.nvfp4_quantize_bf16.restype = i32
        lib.nvfp4_quantize_bf16.argtypes = [P, i64, i64, P, P, P, P, sz, P]
        lib.nvfp4_blocked_scale_bytes.restype = sz
        lib.nvfp4_blocked_scale_bytes.argtypes = [i64, i64]
        lib.nvfp4_import_blocked_scales.restype = i32
        lib.nvfp4_import_blocked_scales.argtypes = [P, i64, i64, P, P]
        lib.nvfp4_fp6_quantize.restype = i32
        lib.nvfp4_fp6_quantize.argtypes = [P, i64, i64, P, P, P]
        lib.nvfp4_fp6_quantize_bf16.restype = i32
        lib.nvfp4_fp6_quantize_bf16.argtypes = [P, i64, i64, P, P, P]
        lib.nvfp4_fp6_gemm.restype = i32
        lib.nvfp4_fp6_gemm.argtypes = [P, i64, P, P, i64, i64, P, i32, P, sz, P]
        lib.nvfp4_fp6_gateup_swiglu.restype = i32
        lib.nvfp4_fp6_gateup_swiglu.argtypes = [P, i64, P, P, P, P, i64, i64, P, i32, P, sz, P]
        lib.nvfp4_gemv_skinny.restype = i32
        lib.nvfp4_gemv_skinny.argtypes = [P, i64, P, P, P, i64, i64, P, i32, P, sz, P]
        lib.nvfp4_gateup_swiglu.restype = i32
        lib.nvfp4_gateup_swiglu.argtypes = [P, i64, P, P, P, P, P, P, i64, i64, P, i32, P, sz, P]
        lib.nvfp4_gemm_prefill.restype = i32
        lib.nvfp4_gemm_prefill.argtypes = [P, i64, P, P, P, i64, i64, P, i32, P, sz, P]
        lib.nvfp4_gemv_skinny_noalloc.restype = i32
        lib.nvfp4_gemv_skinny_noalloc.argtypes = [P, i64, P, P, P, i64, i64, P, i32, P]
        lib.nvfp4_stream_plan_bytes.restype = sz
        lib.nvfp4_stream_plan_bytes.argtypes = [ctypes.POINTER(SkinnyJobC), i32, i64]
        lib.nvfp4_stream_plan.restype = i32
        lib.nvfp4_stream_plan.argtypes = [ctypes.POINTER(SkinnyJobC), i32, i64, P, sz, P]
        lib.nvfp4_stream_run.restype = i32
        lib.nvfp4_stream_run.argtypes = [P, sz, P]
        lib.nvfp4_noalloc_status.restype = i32
        lib.nvfp4_noalloc_status.argtypes = [i32, ctypes.POINTER(ctypes.c_uint32), P]
        lib.nvfp4_noalloc_selftest_wait_timeout.restype = i32
        lib.nvfp4_noalloc_selftest_wait_timeout.argtypes = [P]
        cache_p, args_p = ctypes.POINTER(KVCacheC), ctypes.POINTER(PagedAttentionArgsC)
        lib.nvfp4_kv_page_bytes.restype = sz
        lib.nvfp4_kv_page_bytes.argtypes = [ctypes.c_int32] * 4
        for f in (lib.nvfp4_kv_append, lib.nvfp4_kv_read):
            f.restype = i32
            f.argtypes = [cache_p, P, i64, P, i64, P, i64, P, sz, P]
        lib.nvfp4_paged_attention_workspace_bytes.restype = sz
        lib.nvfp4_paged_attention_workspace_bytes.argtypes = [args_p]
        lib.nvfp4_paged_attention.restype = i32
        lib.nvfp4_paged_attention.argtypes = [args_p, P, sz, P]
        ep_p = ctypes.POINTER(EpilogueC)
        lib.nvfp4_gemm_epilogue.restype = i32
        lib.nvfp4_gemm_epilogue.argtypes = [P, i64, P, P, P, i64, i64, ep_p, P, i32, P, sz, P]
        lib.nvfp4_fp6_gemm_epilogue.restype = i32
        lib.nvfp4_fp6_gemm_epilogue.argtypes = [P, i64, P, P, i64, i64, ep_p, P, i32, P, sz, P]
        lib.nvfp4_rope_pairs.restype = i32
        lib.nvfp4_rope_pairs.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int32), ctypes.c_int32,
                                         P]
        lib.nvfp4_rope.restype = i32
        lib.nvfp4_rope.argtypes = [P, P]  # RopeArgsC, packed
        lib.nvfp4_prompt_attention.restype = i32
        lib.nvfp4_prompt_attention.argtypes = [P, P, sz, P]  # PromptAttentionArgsC, packed
        lib.nvfp4_device_status.restype = i32
        lib.nvfp4_device_status.argtypes = [P, sz, i32, ctypes.POINTER(ctypes.c_uint32), P]
        lib.nvfp4_selftest_wait_timeout.restype = i32
        lib.nvfp4_selftest_wait_timeout.argtypes = [P, sz, P]
        _lib = lib
        return lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/nvfp4.h."""
    text = open(_build.HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(nvfp4_[a-z0-9_]+)\s*\(", text)))


# ---------------------------------------------------------------------------
# Thin wrappers with the C names
# ---------------------------------------------------------------------------

def nvfp4_status_string(status: int) -> str:
    return load_library().nvfp4_status_string(int(status)).decode()


def nvfp4_version() -> int:
    return load_library().nvfp4_version()


def nvfp4_workspace_bytes(op: int, N: int, M: int, K: int) -> int:
    return load_library().nvfp4_workspace_bytes(int(op), int(N), int(M), int(K))


@dataclass
class NVFP4Weight:
    """One NVFP4 tensor W[M][K] in device memory (see include/nvfp4.h)."""
    codes: torch.Tensor         # uint8 [M, K/2]
    scales: torch.Tensor        # uint8 [M, K/16]
    tensor_scale: torch.Tensor  # float32 [1]

    @property
    def M(self) -> int:
        return self.codes.shape[0]

    @property
    def K(self) -> int:
        return self.codes.shape[1] * 2

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != NVFP4_OK:
        raise NVFP4Error(status, where)


def _new(stream, *shape, dtype, device):
    """An output of a call on `stream` (None: the current one): memory of that stream, since nothing orders it behind
    the current one's work, and not given to others before the current one's work so far is done with it."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _zeroed(stream, nbytes, device):
    """A workspace of a call on `stream`, zero-filled there: only that stream's work sees it."""
    if stream is None:
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def _workspace(op, N, M, K, device, workspace, stream):
    need = nvfp4_workspace_bytes(op, N, M, K)
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    if need == 0:
        return None, 0
    # zero-filled: the skinny calls keep split-K counters in it
    return _zeroed(stream, need, device), need


def _out_code(dtype) -> int:
    if dtype == torch.float32:
        return NVFP4_OUT_F32
    if dtype == torch.bfloat16:
        return NVFP4_OUT_BF16
    raise ValueError(f"unsupported output dtype {dtype}")


def nvfp4_quantize(w: torch.Tensor, workspace: torch.Tensor | None = None,
                   out: NVFP4Weight | None = None, stream=None) -> NVFP4Weight:
    """fp32 [M, K] CUDA tensor -> NVFP4Weight (codes, scales, tensor scale)."""
    M, K = w.shape
    if out is None:
        out = NVFP4Weight(_new(stream, M, K // 2, dtype=torch.uint8, device=w.device),
                          _new(stream, M, K // 16, dtype=torch.uint8, device=w.device),
                          _new(stream, 1, dtype=torch.float32, device=w.device))
    ws, ws_bytes = _workspace(NVFP4_OP_QUANTIZE, 0, M, K, w.device, workspace, stream)
    st = load_library().nvfp4_quantize(_ptr(w), M, K, _ptr(out.codes), _ptr(out.scales),
                                       _ptr(out.tensor_scale), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "nvfp4_quantize")
    return out


def nvfp4_quantize_bf16(w: torch.Tensor, workspace: torch.Tensor | None = None,
                        out: NVFP4Weight | None = None, stream=None) -> NVFP4Weight:
    """bf16 [M, K] CUDA tensor -> NVFP4Weight, identical to quantising w.float()."""
    if w.dtype != torch.bfloat16:
        raise ValueError(f"nvfp4_quantize_bf16 takes bf16 weights, got {w.dtype}")
    M, K = w.shape
    if out is None:
        out = NVFP4Weight(_new(stream, M, K // 2, dtype=torch.uint8, device=w.device),
                          _new(stream, M, K // 16, dtype=torch.uint8, device=w.device),
                          _new(stream, 1, dtype=torch.float32, device=w.device))
    ws, ws_bytes = _workspace(NVFP4_OP_QUANTIZE, 0, M, K, w.device, workspace, stream)
    st = load_library().nvfp4_quantize_bf16(_ptr(w), M, K, _ptr(out.codes), _ptr(out.scales),
                                            _ptr(out.tensor_scale), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "nvfp4_quantize_bf16")
    return out


def nvfp4_blocked_scale_bytes(M: int, K: int) -> int:
    return load_library().nvfp4_blocked_scale_bytes(M, K)


def nvfp4_import_blocked_scales(blocked: torch.Tensor, M: int, K: int,
                                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Blocked (128 x 4) E4M3 scale bytes -> row-major uint8 [M, K/16] scales."""
    if blocked.dtype != torch.uint8:
        raise ValueError(f"blocked scales are uint8 bytes, got {blocked.dtype}")
    if blocked.numel() < nvfp4_blocked_scale_bytes(M, K):
        raise ValueError("blocked scale buffer smaller than nvfp4_blocked_scale_bytes(M, K)")
    if out is None:
        out = _new(stream, M, K // 16, dtype=torch.uint8, device=blocked.device)
    st = load_library().nvfp4_import_blocked_scales(_ptr(blocked), M, K, _ptr(out), _stream(stream))
    _check(st, "nvfp4_import_blocked_scales")
    return out


def _new_out(N, M, dtype, device, out, stream):
    return out if out is not None else _new(stream, N, M, dtype=dtype, device=device)


def nvfp4_gemv_skinny(x: torch.Tensor, W: NVFP4Weight, out_dtype=torch.float32,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """y[N, M] = x[N, K] (bf16) . dequant(W)^T for N = 1..16."""
    N, K = x.shape
    y = _new_out(N, W.M, out_dtype, x.device, out, stream)
    ws, ws_bytes = _workspace(NVFP4_OP_GEMV_SKINNY, N, W.M, K, x.device, workspace, stream)
    st = load_library().nvfp4_gemv_skinny(_ptr(x), N, _ptr(W.codes), _ptr(W.scales), _ptr(W.tensor_scale),
                                          W.M, K, _ptr(y), _out_code(y.dtype), _ptr(ws), ws_bytes,
                                          _stream(stream))
    _check(st, "nvfp4_gemv_skinny")
    return y


def nvfp4_gateup_swiglu(x: torch.Tensor, Wg: NVFP4Weight, Wu: NVFP4Weight, out_dtype=torch.float32,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """h[N, M] = silu(x . Wg^T) * (x . Wu^T), any N >= 1."""
    N, K = x.shape
    h = _new_out(N, Wg.M, out_dtype, x.device, out, stream)
    ws, ws_bytes = _workspace(NVFP4_OP_GATEUP_SWIGLU, N, Wg.M, K, x.device, workspace, stream)
    st = load_library().nvfp4_gateup_swiglu(_ptr(x), N, _ptr(Wg.codes), _ptr(Wg.scales),
                                            _ptr(Wg.tensor_scale), _ptr(Wu.codes), _ptr(Wu.scales),
                                            _ptr(Wu.tensor_scale), Wg.M, K, _ptr(h), _out_code(h.dtype),
                                            _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "nvfp4_gateup_swiglu")
    return h


def nvfp4_gemm_prefill(x: torch.Tensor, W: NVFP4Weight, out_dtype=torch.float32,
                       out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """y[N, M] = x[N, K] (bf16) . dequant(W)^T, any N >= 1 (tensor cores for N > 16)."""
    N, K = x.shape
    y = _new_out(N, W.M, out_dtype, x.device, out, stream)
    ws, ws_bytes = _workspace(NVFP4_OP_GEMM_PREFILL, N, W.M, K, x.device, workspace, stream)
    st = load_library().nvfp4_gemm_prefill(_ptr(x), N, _ptr(W.codes), _ptr(W.scales), _ptr(W.tensor_scale),
                                           W.M, K, _ptr(y), _out_code(y.dtype), _ptr(ws), ws_bytes,
                                           _stream(stream))
    _check(st, "nvfp4_gemm_prefill")
    return y


def nvfp4_device_status(workspace: torch.Tensor, clear: bool = True, stream=None) -> tuple[int, int]:
    """(status, code) of the device status word in a product call's workspace:
    (NVFP4_OK, 0), or (NVFP4_ERR_DEVICE_TIMEOUT, code) when a kernel's bounded
    wait gave up since the word was last cleared, or (NVFP4_ERR_DEVICE_INDEX,
    code) when a KV-cache call met an index outside its bounds.  Synchronises the stream;
    with clear=True a nonzero word is reset."""
    code = ctypes.c_uint32(0)
    st = load_library().nvfp4_device_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                            int(bool(clear)), ctypes.byref(code), _stream(stream))
    if st not in (NVFP4_OK, NVFP4_ERR_DEVICE_TIMEOUT, NVFP4_ERR_DEVICE_INDEX):
        raise NVFP4Error(st, "nvfp4_device_status")
    return st, code.value


def nvfp4_selftest_wait_timeout(workspace: torch.Tensor, stream=None) -> None:
    """Enqueue the failure-path self-test: a bounded wait that runs out after
    2 s and records code 127 in the workspace's status word."""
    st = load_library().nvfp4_selftest_wait_timeout(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                                    _stream(stream))
    _check(st, "nvfp4_selftest_wait_timeout")


@dataclass
class FP6Weight:
    """One FP6 E2M3 block-scaled tensor W[M][K] in device memory (include/nvfp4.h)."""
    codes: torch.Tensor   # uint8 [M, 3K/4]
    scales: torch.Tensor  # uint8 [M, K/128] (UE8M0)

    @property
    def M(self) -> int:
        return self.codes.shape[0]

    @property
    def K(self) -> int:
        return self.codes.shape[1] // 6 * 8

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _fp6_out(M, K, device, out, stream):
    if out is not None:
        return out
    return FP6Weight(_new(stream, M, K // 8 * 6, dtype=torch.uint8, device=device),
                     _new(stream, M, K // 128, dtype=torch.uint8, device=device))


def nvfp4_fp6_quantize(w: torch.Tensor, out: FP6Weight | None = None, stream=None) -> FP6Weight:
    """fp32 [M, K] CUDA tensor (K % 128 == 0) -> FP6Weight."""
    if w.dtype != torch.float32:
        raise ValueError(f"nvfp4_fp6_quantize takes fp32 weights, got {w.dtype}")
    M, K = w.shape
    out = _fp6_out(M, K, w.device, out, stream)
    st = load_library().nvfp4_fp6_quantize(_ptr(w), M, K, _ptr(out.codes), _ptr(out.scales), _stream(stream))
    _check(st, "nvfp4_fp6_quantize")
    return out


def nvfp4_fp6_quantize_bf16(w: torch.Tensor, out: FP6Weight | None = None, stream=None) -> FP6Weight:
    """bf16 [M, K] CUDA tensor -> FP6Weight, identical to quantising w.float()."""
    if w.dtype != torch.bfloat16:
        raise ValueError(f"nvfp4_fp6_quantize_bf16 takes bf16 weights, got {w.dtype}")
    M, K = w.shape
    out = _fp6_out(M, K, w.device, out, stream)
    st = load_library().nvfp4_fp6_quantize_bf16(_ptr(w), M, K, _ptr(out.codes), _ptr(out.scales),
                                                _stream(stream))
    _check(st, "nvfp4_fp6_quantize_bf16")
    return out


def nvfp4_fp6_gemm(x: torch.Tensor, W: FP6Weight, out_dtype=torch.float32, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[N, M] = x[N, K] (bf16) . dequant(W)^T for FP6 weights, any N >= 1."""
    N, K = x.shape
    y = _new_out(N, W.M, out_dtype, x.device, out, stream)
    ws, ws_bytes = _workspace(NVFP4_OP_FP6_GEMM, N, W.M, K, x.device, workspace, stream)
    st = load_library().nvfp4_fp6_gemm(_ptr(x), N, _ptr(W.codes), _ptr(W.scales), W.M, K, _ptr(y),
                                       _out_code(y.dtype), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "nvfp4_fp6_gemm")
    return y


def nvfp4_fp6_gateup_swiglu(x: torch.Tensor, Wg: FP6Weight, Wu: FP6Weight, out_dtype=torch.float32,
                            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """h[N, M] = silu(x . Wg^T) * (x . Wu^T) for FP6 weights, any N >= 1."""
    N, K = x.shape
    h = _new_out(N, Wg.M, out_dtype, x.device, out, stream)
    ws, ws_bytes = _workspace(NVFP4_OP_FP6_GATEUP_SWIGLU, N, Wg.M, K, x.device, workspace, stream)
    st = load_library().nvfp4_fp6_gateup_swiglu(_ptr(x), N, _ptr(Wg.codes), _ptr(Wg.scales), _ptr(Wu.codes),
                                                _ptr(Wu.scales), Wg.M, K, _ptr(h), _out_code(h.dtype),
                                                _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "nvfp4_fp6_gateup_swiglu")
    return h


def nvfp4_gemv_skinny_noalloc(x: torch.Tensor, W: NVFP4Weight, out_dtype=torch.float32,
                              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Skinny product whose scratch is the library's fixed device array (for
    callers that cannot allocate device memory; see include/nvfp4.h).  The
    output tensor is the only buffer created here, and only when `out` is None."""
    N, K = x.shape
    y = _new_out(N, W.M, out_dtype, x.device, out, stream)
    st = load_library().nvfp4_gemv_skinny_noalloc(_ptr(x), N, _ptr(W.codes), _ptr(W.scales),
                                                  _ptr(W.tensor_scale), W.M, K, _ptr(y),
                                                  _out_code(y.dtype), _stream(stream))
    _check(st, "nvfp4_gemv_skinny_noalloc")
    return y


def nvfp4_noalloc_status(clear: bool = True, stream=None) -> tuple[int, int]:
    """(status, code) of the status word in the no-allocation array of the
    current device; with clear=True a nonzero word zero-fills the array."""
    code = ctypes.c_uint32(0)
    st = load_library().nvfp4_noalloc_status(int(bool(clear)), ctypes.byref(code), _stream(stream))
    if st not in (NVFP4_OK, NVFP4_ERR_DEVICE_TIMEOUT):
        raise NVFP4Error(st, "nvfp4_noalloc_status")
    return st, code.value


def nvfp4_noalloc_selftest_wait_timeout(stream=None) -> None:
    """Enqueue the bounded-wait self-test against the no-allocation array."""
    _check(load_library().nvfp4_noalloc_selftest_wait_timeout(_stream(stream)),
           "nvfp4_noalloc_selftest_wait_timeout")


# ---------------------------------------------------------------------------
# Product lists in one launch (nvfp4_stream_plan / nvfp4_stream_run)
# ---------------------------------------------------------------------------

@dataclass
class SkinnyJob:
    """One product of a list: y = x . W^T, or silu(x . Wg^T) * (x . Wu^T) when
    W is a (gate, up) pair.  x is a bf16 [N, K] tensor (rows may be strided),
    or None with `input` the index of an earlier job whose bf16 output is x."""
    W: object                       # NVFP4Weight, or (gate, up) NVFP4Weights
    y: torch.Tensor                 # [N, M] float32 or bfloat16
    x: torch.Tensor | None = None
    input: int = -1

    def weights(self):
        return list(self.W) if isinstance(self.W, (tuple, list)) else [self.W]


def _job_structs(jobs):
    arr = (SkinnyJobC * len(jobs))()
    for i, j in enumerate(jobs):
        ws = j.weights()
        c = arr[i]
        if j.x is not None:
            if j.x.dtype != torch.bfloat16 or j.x.stride(1) != 1:
                raise ValueError("job activations must be bf16 with unit stride along K")
            c.x = j.x.data_ptr()
            c.x_ld = j.x.stride(0)
        c.input = int(j.input)
        c.n_weights = len(ws)
        for k, W in enumerate(ws):
            c.codes[k] = W.codes.data_ptr()
            c.scales[k] = W.scales.data_ptr()
            c.tensor_scale[k] = W.tensor_scale.data_ptr()
        c.M = ws[0].M
        c.K = ws[0].K
        c.y = j.y.data_ptr()
        c.out_dtype = _out_code(j.y.dtype)
    return arr


class StreamPlan:
    """A plan buffer (device) and the tensors its jobs point to (kept alive)."""

    def __init__(self, buffer: torch.Tensor, jobs, N: int):
        self.buffer = buffer
        self.jobs = list(jobs)
        self.N = N

    def nbytes(self) -> int:
        return self.buffer.numel()


def nvfp4_stream_plan_bytes(jobs, N: int) -> int:
    arr = _job_structs(jobs)
    return load_library().nvfp4_stream_plan_bytes(arr, len(jobs), int(N))


def nvfp4_stream_plan(jobs, N: int, device=None, stream=None) -> StreamPlan:
    """Build the device plan of a job list (synchronises the stream)."""
    arr = _job_structs(jobs)
    lib = load_library()
    need = lib.nvfp4_stream_plan_bytes(arr, len(jobs), int(N))
    if need == 0:
        raise NVFP4Error(NVFP4_ERR_INVALID_ARG, "nvfp4_stream_plan_bytes")
    dev = device or jobs[0].y.device
    buf = _new(stream, need, dtype=torch.uint8, device=dev)
    st = lib.nvfp4_stream_plan(arr, len(jobs), int(N), _ptr(buf), need, _stream(stream))
    _check(st, "nvfp4_stream_plan")
    return StreamPlan(buf, jobs, int(N))


def nvfp4_stream_run(plan: StreamPlan, stream=None) -> None:
    """Run every job of a plan (one launch, asynchronous)."""
    st = load_library().nvfp4_stream_run(_ptr(plan.buffer), plan.nbytes(), _stream(stream))
    _check(st, "nvfp4_stream_run")



# ---------------------------------------------------------------------------
# Quantised paged KV cache and attention over it
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def nvfp4_kv_page_bytes(page_size: int, n_kv_heads: int, head_dim: int, format: int) -> int:
    return load_library().nvfp4_kv_page_bytes(page_size, n_kv_heads, head_dim, format)


# Handle of the current stream without a Stream object around it: these calls
# take a few microseconds, and making that object is one or two of them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
@functools.lru_cache(maxsize=1)
def _one_gpu() -> bool:
    return torch.cuda.device_count() == 1


def _on_device_of(where, *tensors):
    """Makes the device of the tensors (those that are not None) current; they must share one CUDA device.  (The calls
    come here only where being CUDA tensors does not settle it: looking at eight devices takes a microsecond.)"""
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1 or next(iter(devices)).type != "cuda":
        raise ValueError(f"{where}: all tensors must be on one CUDA device, got {', '.join(sorted(map(str, devices)))}")
    return torch.cuda.device(devices.pop())


def _stream_of(t: torch.Tensor, stream) -> int:
    """Stream handle: `stream`, or the current one of the device that holds t."""
    if stream is not None:
        return stream.cuda_stream
    device = t.get_device()
    if device < 0:
        return None  # not a CUDA tensor: refused before anything is launched
    return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(t.device).cuda_stream


@dataclass
class KVCache:
    """One layer's quantised paged KV cache (include/nvfp4.h has the layout)."""
    pool: torch.Tensor   # uint8 [n_pages, n_kv_heads, 2 (K, V), block]
    page_size: int       # tokens of a page: 16, 32, 64, 128 or 256
    head_dim: int        # 64 or 128
    format: int          # NVFP4_KV_E4M3 or NVFP4_KV_NVFP4

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, format: int = NVFP4_KV_E4M3,
              device="cuda") -> "KVCache":
        """A cache of n_pages pages; its slots hold nothing until they are appended to."""
        size = nvfp4_kv_page_bytes(page_size, n_kv_heads, head_dim, format)
        if size == 0:
            raise NVFP4Error(NVFP4_ERR_UNSUPPORTED_SHAPE, "KVCache.empty")
        return cls(torch.empty(n_pages, n_kv_heads, 2, size // (2 * n_kv_heads), dtype=torch.uint8, device=device),
                   page_size, head_dim, format)

    @property
    def n_pages(self) -> int:
        return self.pool.shape[0]

    @property
    def n_kv_heads(self) -> int:
        return self.pool.shape[1]

    def c(self) -> KVCacheC:
        pool = self.pool
        n_pages, heads = pool.shape[0], pool.shape[1]
        if pool.dtype != torch.uint8 or not pool.is_contiguous() or pool.numel() != n_pages * nvfp4_kv_page_bytes(
                self.page_size, heads, self.head_dim, self.format):
            raise ValueError("pool is not a contiguous uint8 [n_pages, n_kv_heads, 2, block] of this cache's format")
        return KVCacheC(pool.data_ptr(), n_pages, self.page_size, heads, self.head_dim, self.format)


def _buffer(t):
    """(address, bytes) of a workspace tensor, or of none."""
    return (None, 0) if t is None else (t.data_ptr(), t.numel() * t.element_size())


def _head_rows(t, heads, head_dim, dtypes, what):
    """Token stride (elements) of [tokens, heads, head_dim] rows whose heads lie side by side."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim or t.dtype not in dtypes:
        raise ValueError(f"{what} must be {' or '.join(str(d) for d in dtypes)} [tokens, {heads}, {head_dim}], "
                         f"got {t.dtype} {list(shape)}")
    if stride[2] != 1 or (heads > 1 and stride[1] != head_dim):
        raise ValueError(f"{what}: the heads of a token must lie side by side (strides {stride})")
    return stride[0] if shape[0] > 1 else heads * head_dim  # one token's stride is never used


_BF16 = (torch.bfloat16,)


def _token_rows(t, tokens, heads, head_dim, dtype, what):
    """Token stride (elements) of `tokens` such rows of one type."""
    if t.is_contiguous() and t.dtype is dtype and t.shape == (tokens, heads, head_dim):
        return heads * head_dim
    ld = _head_rows(t, heads, head_dim, (dtype,), what)
    if t.shape[0] != tokens:
        raise ValueError(f"{what} has {t.shape[0]} tokens, not {tokens}")
    return ld


# Argument blocks of calls that take a few microseconds, field by field as in their ctypes.Structure (making one of
# those takes longer than the rest of the call).
_ROPE_ARGS = struct.Struct("@PPqqPPqqPqPqiiiiiiiifi")
_PROMPT_ARGS = struct.Struct("@PPPqqqPqPqqqiiiiif")


def _check_slots(slots, tokens):
    if slots.dtype != torch.int64 or slots.shape != (tokens,) or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int64 [{tokens}], got {slots.dtype} {list(slots.shape)}")


def nvfp4_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    workspace: torch.Tensor | None = None, stream=None) -> None:
    """Quantise bf16 k, v [tokens, n_kv_heads, head_dim] (token rows may be
    strided, as column ranges of a QKV output are) into the cache's slots.  A
    negative slot leaves its token out."""
    c = cache.c()
    k_ld = _head_rows(k, c.n_kv_heads, c.head_dim, _BF16, "k")
    v_ld = _head_rows(v, c.n_kv_heads, c.head_dim, _BF16, "v")
    if v.shape[0] != k.shape[0]:
        raise ValueError(f"k has {k.shape[0]} tokens, v {v.shape[0]}")
    _check_slots(slots, k.shape[0])
    ws, ws_bytes = _buffer(workspace)
    args = (ctypes.byref(c), k.data_ptr(), k_ld, v.data_ptr(), v_ld, slots.data_ptr(), k.shape[0], ws, ws_bytes,
            _stream_of(slots, stream))
    if (slots.is_cuda and cache.pool.is_cuda and k.is_cuda and v.is_cuda and (workspace is None or workspace.is_cuda)
            and _one_gpu()):
        st = load_library().nvfp4_kv_append(*args)
    else:
        with _on_device_of("nvfp4_kv_append", slots, cache.pool, k, v, workspace):
            st = load_library().nvfp4_kv_append(*args)
    if st:
        _check(st, "nvfp4_kv_append")


def nvfp4_kv_read(cache: KVCache, slots: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(k, v) of the cache's slots as bf16 [tokens, n_kv_heads, head_dim]; rows
    of negative slots are zero."""
    c = cache.c()
    if out is None:
        out = tuple(_new(stream, slots.numel(), c.n_kv_heads, c.head_dim, dtype=torch.bfloat16, device=slots.device)
                    for _ in range(2))
    k, v = out
    k_ld = _head_rows(k, c.n_kv_heads, c.head_dim, _BF16, "k")
    v_ld = _head_rows(v, c.n_kv_heads, c.head_dim, _BF16, "v")
    _check_slots(slots, k.shape[0])
    _check_slots(slots, v.shape[0])
    ws, ws_bytes = _buffer(workspace)
    args = (ctypes.byref(c), k.data_ptr(), k_ld, v.data_ptr(), v_ld, slots.data_ptr(), k.shape[0], ws, ws_bytes,
            _stream_of(slots, stream))
    if (slots.is_cuda and cache.pool.is_cuda and k.is_cuda and v.is_cuda and (workspace is None or workspace.is_cuda)
            and _one_gpu()):
        st = load_library().nvfp4_kv_read(*args)
    else:
        with _on_device_of("nvfp4_kv_read", slots, cache.pool, k, v, workspace):
            st = load_library().nvfp4_kv_read(*args)
    if st:
        _check(st, "nvfp4_kv_read")
    return out


def nvfp4_paged_attention_workspace_bytes(cache: KVCache, q: torch.Tensor, n_seqs: int, max_q_len: int) -> int:
    """Bytes of workspace for attention of q [total_q, n_q_heads, head_dim] over the cache."""
    a = PagedAttentionArgsC(cache=cache.c(), n_seqs=n_seqs, total_q=q.shape[0], max_q_len=max_q_len,
                            n_q_heads=q.shape[1])
    return load_library().nvfp4_paged_attention_workspace_bytes(ctypes.byref(a))


def _device_ints(t, dtype, shape, what):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def nvfp4_paged_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                          q_offsets: torch.Tensor | None = None, max_q_len: int | None = None,
                          scale: float | None = None, causal: bool = True, window: int = 0,
                          tree: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Attention of new tokens q (bf16 [total_q, n_q_heads, head_dim]) over the cache.

    block_table int32 [n_seqs, width] (contiguous, as the other index tensors), kv_lens int32 [n_seqs] (keys in the
    cache, the new tokens' own among them when causal); q_offsets int32
    [n_seqs + 1] for sequences with different numbers of new tokens, with
    max_q_len their largest; tree int64 [total_q], bit j of a token's word:
    it sees the sequence's new token j.  scale defaults to head_dim ** -0.5."""
    c = cache.c()
    if q.dim() != 3:
        raise ValueError(f"q must be [total_q, n_q_heads, head_dim], got {list(q.shape)}")
    total_q, heads, head_dim = q.shape
    q_ld = _head_rows(q, heads, c.head_dim, _BF16, "q")
    n_seqs = kv_lens.shape[0]
    if block_table.dim() != 2:
        raise ValueError(f"block_table must be [n_seqs, width], got {list(block_table.shape)}")
    width = block_table.shape[1]
    if max_q_len is None:
        if q_offsets is not None:
            raise ValueError("q_offsets needs max_q_len")
        if n_seqs == 0 or total_q % n_seqs:
            raise ValueError(f"{total_q} tokens are not the same number for each of {n_seqs} sequences: give q_offsets")
        max_q_len = total_q // n_seqs
    if out is None:
        out = _new(stream, total_q, heads, head_dim, dtype=out_dtype, device=q.device)
    out_ld = _head_rows(out, heads, c.head_dim, (torch.bfloat16, torch.float32), "out")
    if out.shape[0] != total_q:
        raise ValueError(f"q has {total_q} tokens, out {out.shape[0]}")
    a = PagedAttentionArgsC(
        c, q.data_ptr(), q_ld, out.data_ptr(), out_ld,
        _device_ints(block_table, torch.int32, (n_seqs, width), "block_table"), width,
        _device_ints(kv_lens, torch.int32, (n_seqs,), "kv_lens"),
        None if q_offsets is None else _device_ints(q_offsets, torch.int32, (n_seqs + 1,), "q_offsets"),
        None if tree is None else _device_ints(tree, torch.int64, (total_q,), "tree"),
        n_seqs, total_q, max_q_len, window, heads, _out_code(out.dtype), 1 if causal else 0,
        head_dim ** -0.5 if scale is None else scale)
    lib = load_library()
    if workspace is None:
        # zero-filled: the call keeps arrival counters in it
        workspace = _zeroed(stream, lib.nvfp4_paged_attention_workspace_bytes(ctypes.byref(a)), q.device)
    ws, ws_bytes = _buffer(workspace)
    args = (ctypes.byref(a), ws, ws_bytes, _stream_of(q, stream))
    if (q.is_cuda and cache.pool.is_cuda and block_table.is_cuda and kv_lens.is_cuda and out.is_cuda and workspace.is_cuda
            and (q_offsets is None or q_offsets.is_cuda) and (tree is None or tree.is_cuda) and _one_gpu()):
        st = lib.nvfp4_paged_attention(*args)
    else:
        with _on_device_of("nvfp4_paged_attention", q, cache.pool, block_table, kv_lens, q_offsets, tree, out, workspace):
            st = lib.nvfp4_paged_attention(*args)
    if st:
        _check(st, "nvfp4_paged_attention")
    return out


# ---------------------------------------------------------------------------
# Products with an epilogue
# ---------------------------------------------------------------------------

def _product_epilogue(where, call, op, x, M, K, weight, bias, activation, residual, out_dtype, out, workspace, stream):
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != K or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous bf16 [tokens, {K}], got {x.dtype} {list(x.shape)}")
    N = x.shape[0]
    if bias is not None and (bias.shape != (M,) or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous [{M}], got {list(bias.shape)}")
    if residual is not None and (residual.shape != (N, M) or (M > 1 and residual.stride(1) != 1)):
        raise ValueError(f"residual must be [{N}, {M}] with unit stride along its rows, got {list(residual.shape)}")
    if out is None:
        out = _new(stream, N, M, dtype=out_dtype, device=x.device)
    if out.shape != (N, M) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous [{N}, {M}], got {list(out.shape)}")
    e = EpilogueC(None if bias is None else bias.data_ptr(), None if residual is None else residual.data_ptr(),
                  0 if residual is None else (residual.stride(0) if N > 1 else M),
                  0 if bias is None else _out_code(bias.dtype), 0 if residual is None else _out_code(residual.dtype),
                  activation, 0)
    if workspace is None:
        # zero-filled: the calls with few tokens keep split-K counters in it
        workspace = _zeroed(stream, max(16, nvfp4_workspace_bytes(op, N, M, K)), x.device)
    ws, ws_bytes = _buffer(workspace)
    args = (x.data_ptr(), N, *(t.data_ptr() for t in weight), M, K, ctypes.byref(e), out.data_ptr(), _out_code(out.dtype),
            ws, ws_bytes, _stream_of(x, stream))
    if (x.is_cuda and out.is_cuda and workspace.is_cuda and all(t.is_cuda for t in weight)
            and (bias is None or bias.is_cuda) and (residual is None or residual.is_cuda) and _one_gpu()):
        st = call(*args)
    else:
        with _on_device_of(where, x, *weight, bias, residual, out, workspace):
            st = call(*args)
    if st:
        _check(st, where)
    return out


def nvfp4_gemm_epilogue(x: torch.Tensor, W: NVFP4Weight, bias: torch.Tensor | None = None,
                        activation: int = NVFP4_ACT_NONE, residual: torch.Tensor | None = None, out_dtype=torch.float32,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """y[N, M] = residual + act(x[N, K] (bf16) . dequant(W)^T + bias), any N >= 1; bias [M] and residual [N, M] (rows may
    be strided) bf16 or fp32; `out` may be the residual itself."""
    return _product_epilogue("nvfp4_gemm_epilogue", load_library().nvfp4_gemm_epilogue, NVFP4_OP_GEMM_PREFILL, x, W.M, W.K,
                             (W.codes, W.scales, W.tensor_scale), bias, activation, residual, out_dtype, out, workspace, stream)


def nvfp4_fp6_gemm_epilogue(x: torch.Tensor, W: FP6Weight, bias: torch.Tensor | None = None,
                            activation: int = NVFP4_ACT_NONE, residual: torch.Tensor | None = None,
                            out_dtype=torch.float32, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_gemm_epilogue for FP6 weights."""
    return _product_epilogue("nvfp4_fp6_gemm_epilogue", load_library().nvfp4_fp6_gemm_epilogue, NVFP4_OP_FP6_GEMM, x, W.M,
                             W.K, (W.codes, W.scales), bias, activation, residual, out_dtype, out, workspace, stream)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def nvfp4_rope_pairs(inv_freq, axis=None) -> torch.Tensor:
    """Table entries (a CPU uint8 [n_pairs, 16]) for frequencies in radians per position (a sequence or a 1-D tensor,
    taken as fp64) and each pair's axis (all 0 without)."""
    freq = [float(f) for f in inv_freq]
    n = len(freq)
    if axis is not None and len(axis) != n:
        raise ValueError(f"{n} frequencies, {len(axis)} axes")
    pairs = torch.zeros(n, 16, dtype=torch.uint8)
    axes = None if axis is None else (ctypes.c_int32 * n)(*(int(a) for a in axis))
    st = load_library().nvfp4_rope_pairs((ctypes.c_double * n)(*freq), axes, n, pairs.data_ptr())
    _check(st, "nvfp4_rope_pairs")
    return pairs


@dataclass
class RopeTable:
    """Each pair's frequency and axis in device memory (include/nvfp4.h), made once for a model."""
    pairs: torch.Tensor  # uint8 [n_pairs, 16]
    n_axes: int          # axes that the pairs use: positions need as many rows

    @classmethod
    def make(cls, inv_freq, axis=None, device="cuda") -> "RopeTable":
        """inv_freq: radians per position of each pair, e.g. base ** (-2 * i / rotary_dim); axis: each pair's row of the
        positions (all 0 without)."""
        pairs = nvfp4_rope_pairs(inv_freq, axis)
        return cls(pairs.to(device), 1 + (max((int(a) for a in axis), default=0) if axis is not None else 0))

    @property
    def n_pairs(self) -> int:
        return self.pairs.shape[0]


def nvfp4_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, table: RopeTable,
               adjacent: bool = False, inverse: bool = False, scale: float = 1.0,
               out: tuple[torch.Tensor, torch.Tensor | None] | None = None,
               stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(q, k) turned by their tokens' positions.

    q [tokens, n_q_heads, head_dim] and k [tokens, n_k_heads, head_dim] (or None), both bf16 or fp32, token rows may be
    strided; positions int64 [tokens], or [axes, tokens] for a table with several axes (text, whose tokens have one
    position for all axes, may pass positions.expand(axes, -1)).  out: two tensors of the
    inputs' shapes and type, which may be the inputs themselves (in place)."""
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim], got {list(shape)}")
    tokens, heads, head_dim = shape
    code = _out_code(dtype)
    k_heads = 0
    if k is not None:
        if k.dim() != 3:
            raise ValueError(f"k must be [tokens, heads, head_dim], got {list(k.shape)}")
        k_heads = k.shape[1]
    if out is None:
        out = (_new(stream, tokens, heads, head_dim, dtype=dtype, device=q.device),
               None if k is None else _new(stream, tokens, k_heads, head_dim, dtype=dtype, device=q.device))
    q_out, k_out = out
    if (k is None) != (k_out is None):
        raise ValueError("out must hold a tensor for k if and only if k is given")
    q_ld = _token_rows(q, tokens, heads, head_dim, dtype, "q")
    q_out_ld = _token_rows(q_out, tokens, heads, head_dim, dtype, "out[0]")
    k_ptr = k_out_ptr = k_ld = k_out_ld = 0
    if k is not None:
        k_ld = _token_rows(k, tokens, k_heads, head_dim, dtype, "k")
        k_out_ld = _token_rows(k_out, tokens, k_heads, head_dim, dtype, "out[1]")
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    at = positions.shape
    axes = at[0] if len(at) == 2 else 1
    if positions.dtype is not torch.int64 or len(at) not in (1, 2) or at[-1] != tokens or (
            not positions.is_contiguous() and tokens > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions must be int64 [{tokens}] or [axes, {tokens}] with unit stride along the tokens, got "
                         f"{positions.dtype} {list(at)}")
    if axes < table.n_axes:
        raise ValueError(f"the table uses {table.n_axes} axes, positions have {axes}")
    pairs = table.pairs
    n_pairs = pairs.shape[0]
    if pairs.dtype is not torch.uint8 or pairs.shape != (n_pairs, 16) or not pairs.is_contiguous():
        raise ValueError(f"the table's pairs must be a contiguous uint8 [n_pairs, 16], got {pairs.dtype} {list(pairs.shape)}")
    a = _ROPE_ARGS.pack(q.data_ptr(), k_ptr, q_ld, k_ld, q_out.data_ptr(), k_out_ptr, q_out_ld, k_out_ld, positions.data_ptr(),
                        positions.stride(0) if axes > 1 else tokens, pairs.data_ptr(), tokens, axes, n_pairs, heads, k_heads,
                        head_dim, code, 1 if adjacent else 0, 1 if inverse else 0, scale, 0)
    s = _stream_of(q, stream)
    if (q.is_cuda and q_out.is_cuda and positions.is_cuda and pairs.is_cuda and (k is None or (k.is_cuda and k_out.is_cuda))
            and _one_gpu()):
        st = load_library().nvfp4_rope(a, s)
    else:
        with _on_device_of("nvfp4_rope", q, q_out, k, k_out, positions, pairs):
            st = load_library().nvfp4_rope(a, s)
    if st:
        _check(st, "nvfp4_rope")
    return out


# ---------------------------------------------------------------------------
# Attention over whole prompts
# ---------------------------------------------------------------------------

def nvfp4_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor | None = None,
                           scale: float | None = None, causal: bool = True, window: int = 0, out_dtype=torch.bfloat16,
                           out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """Attention of packed prompts over their own K and V.

    q bf16 [tokens, n_q_heads, head_dim], k and v bf16 [tokens, n_kv_heads, head_dim] (token rows may be strided, as
    column ranges of a QKV output are); offsets int32 [n_seqs + 1]: where each sequence begins and the last one ends
    (None: one sequence).  scale defaults to head_dim ** -0.5.  Rows of `out` that belong to no sequence are left as
    they are."""
    shape = q.shape
    if len(shape) != 3 or k.dim() != 3:
        raise ValueError(f"q and k must be [tokens, heads, head_dim], got {list(shape)} and {list(k.shape)}")
    total, heads, head_dim = shape
    kv_heads = k.shape[1]
    q_ld = _token_rows(q, total, heads, head_dim, torch.bfloat16, "q")
    k_ld = _token_rows(k, total, kv_heads, head_dim, torch.bfloat16, "k")
    v_ld = _token_rows(v, total, kv_heads, head_dim, torch.bfloat16, "v")
    if out is None:
        out = _new(stream, total, heads, head_dim, dtype=out_dtype, device=q.device)
    if out.dtype is not torch.bfloat16 and out.dtype is not torch.float32:
        _head_rows(out, heads, head_dim, (torch.bfloat16, torch.float32), "out")  # raises
    code = _out_code(out.dtype)
    out_ld = _token_rows(out, total, heads, head_dim, out.dtype, "out")
    n_seqs, off = 1, 0
    if offsets is not None:
        if offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError(f"offsets must be [n_seqs + 1], got {list(offsets.shape)}")
        n_seqs = offsets.shape[0] - 1
        off = _device_ints(offsets, torch.int32, (n_seqs + 1,), "offsets")
    a = _PROMPT_ARGS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_ld, k_ld, v_ld, out.data_ptr(), out_ld, off, n_seqs, total,
                          window, heads, kv_heads, head_dim, code, 1 if causal else 0,
                          head_dim ** -0.5 if scale is None else scale)
    ws, ws_bytes = _buffer(workspace)
    s = _stream_of(q, stream)
    if (q.is_cuda and k.is_cuda and v.is_cuda and out.is_cuda and (offsets is None or offsets.is_cuda)
            and (workspace is None or workspace.is_cuda) and _one_gpu()):
        st = load_library().nvfp4_prompt_attention(a, ws, ws_bytes, s)
    else:
        with _on_device_of("nvfp4_prompt_attention", q, k, v, out, offsets, workspace):
            st = load_library().nvfp4_prompt_attention(a, ws, ws_bytes, s)
    if st:
        _check(st, "nvfp4_prompt_attention")
    return out
