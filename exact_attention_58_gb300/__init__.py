"""Fused exact attention for GB300 (sm_103a): Python binding of libgbattn.so.

The functions here carry the names of the C ABI in ``include/gbattn.h`` and
do argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libgbattn.so``.  PyTorch supplies device memory and streams.
There is no fallback: if the library has not been built, or an argument is
unsupported, the call raises.

    import exact_attention_58_gb300 as ea
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    dq, dk, dv = ea.attn_bwd(q, k, v, o, do, lse, causal=True)

q, o, do, dq are [B, H, N, d] and k, v, dk, dv [B, H, Nk, d] (Nk = N for
self-attention), contiguous, on one CUDA device; bf16 or fp16 (d = 64 or 128;
the forward also d = 256), or, forward only, fp32 with d = 64 and e4m3
(torch.float8_e4m3fn, O in bf16) with d = 128.  attn_fwd_varlen and
attn_bwd_varlen take packed sequences: [total, H, d] tensors and cumulative
offsets.

Serving from a paged key/value cache (bf16 or fp16, grouped query heads):

    cu, seq_lens, slots, taken = ea.attn_page_table(cached_lens, new_lens, page_table,
                                                    free_pages, num_free, page_size, max_tokens)
    ea.attn_cache_append(k, v, k_cache, v_cache, slots)
    o, lse = ea.attn_fwd_paged(q, k_cache, v_cache, page_table, seq_lens, cu, max_seqlen_q,
                               causal=True)

With rotary positions the step's append rotates too, and a cache of e4m3 values
(torch.float8_e4m3fn) has float32 scales per page and head, powers of two:

    q = ea.attn_cache_append_rope(q, k, v, k_cache, v_cache, slots, inv_freq,
                                  cu_seqlens_q=cu, seq_lens=seq_lens)
    q, k = ea.attn_rope(q, k, inv_freq, positions)
    ea.attn_cache_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, slots)
    o, lse = ea.attn_fwd_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                   cu, max_seqlen_q, causal=True)
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import threading
from typing import Optional

import torch

from . import _build

__all__ = [
    "AttnError", "attn_fwd", "attn_bwd", "attn_bwd_workspace_size", "attn_bwd_preprocess",
    "attn_bwd_main", "attn_bwd_dq_convert", "attn_bwd_noalloc", "attn_fwd_varlen",
    "attn_bwd_varlen", "attn_page_table", "attn_cache_append", "attn_fwd_paged",
    "attn_fwd_paged_workspace_size", "attn_rope", "attn_rope_frequencies",
    "attn_cache_append_rope", "attn_cache_append_fp8", "attn_fwd_paged_fp8",
    "attn_selftest_wait", "attn_selftest_fwd_withheld", "attn_status_string",
    "attn_version", "library",
    "LIB_PATH", "STATUS",
]

LIB_PATH = _build.LIB_PATH

STATUS = {
    0: "ATTN_OK",
    1: "ATTN_ERR_INVALID_ARG",
    2: "ATTN_ERR_UNSUPPORTED",
    3: "ATTN_ERR_MISALIGNED",
    4: "ATTN_ERR_WORKSPACE",
    5: "ATTN_ERR_CUDA",
    6: "ATTN_ERR_DEVICE_TIMEOUT",
}
_DTYPE = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
if hasattr(torch, "float8_e4m3fn"):
    _DTYPE[torch.float8_e4m3fn] = 3


def _out_dtype(q: torch.Tensor):
    """O takes q's dtype, except bf16 for e4m3 inputs."""
    return torch.bfloat16 if _DTYPE.get(q.dtype) == 3 else q.dtype

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    """A non-zero attn_status from the library."""

    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, self.status)} "
                         f"({attn_status_string(self.status)})")


def library():
    """The loaded libgbattn.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with exact_attention_58_gb300._build.build() "
                    "(there is no fallback implementation)")
            lib = ctypes.CDLL(LIB_PATH)
            vp, ip, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            f, u64 = ctypes.c_float, ctypes.c_uint64
            lib.attn_fwd.argtypes = [vp] * 5 + [ip] * 6 + [f, ip, ip, vp, f, u64, vp, vp]
            lib.attn_bwd.argtypes = [vp] * 9 + [ip] * 6 + [f, ip, ip, vp, f, u64, vp, sz, vp, vp]
            lib.attn_bwd_noalloc.argtypes = [vp] * 9 + [ip] * 6 + [f, ip, ip, vp, f, u64, vp, vp]
            lib.attn_bwd_workspace_size.argtypes = [ip, ip, ip, ip]
            lib.attn_bwd_workspace_size.restype = sz
            lib.attn_bwd_preprocess.argtypes = [vp, vp, vp, ip, ip, ip, ip, ip, vp, sz, vp]
            lib.attn_bwd_main.argtypes = [vp] * 6 + [ip] * 6 + [f, ip, ip, vp, f, u64, vp, sz, vp,
                                                              vp]
            lib.attn_bwd_dq_convert.argtypes = [vp, ip, ip, ip, ip, ip, f, vp, sz, vp]
            lib.attn_fwd_varlen.argtypes = [vp] * 7 + [ip] * 8 + [f, ip, ip, f, u64, vp, vp]
            lib.attn_selftest_wait.argtypes = [vp, ip, vp]
            lib.attn_selftest_wait.restype = ctypes.c_int
            lib.attn_selftest_fwd_withheld.argtypes = [vp] * 5 + [ip] * 6 + [vp, vp]
            lib.attn_selftest_fwd_withheld.restype = ctypes.c_int
            lib.attn_bwd_varlen.argtypes = ([vp] * 11 + [ip] * 8 +
                                            [f, ip, ip, f, u64, vp, sz, vp, vp])
            i64 = ctypes.c_int64
            lib.attn_page_table.argtypes = [vp] * 9 + [ip] * 5 + [vp, vp]
            lib.attn_cache_append.argtypes = ([vp] * 5 + [ip] * 4 + [i64] * 2 + [ip] * 2 +
                                              [i64] * 3 + [vp, vp])
            lib.attn_fwd_paged.argtypes = ([vp] * 8 + [ip] * 10 + [i64] * 5 +
                                           [f, ip, ip, vp, sz, vp, vp])
            lib.attn_rope.argtypes = [vp] * 6 + [ip] * 7 + [i64] * 13 + [f, ip, ip, vp]
            lib.attn_cache_append_rope.argtypes = ([vp] * 11 + [ip] * 7 + [i64] * 6 + [ip] * 2 +
                                                   [i64] * 3 + [f, ip, vp, vp])
            lib.attn_cache_append_fp8.argtypes = ([vp] * 7 + [ip] * 4 + [i64] * 2 + [ip] * 2 +
                                                  [i64] * 3 + [vp, vp])
            lib.attn_fwd_paged_fp8.argtypes = ([vp] * 10 + [ip] * 10 + [i64] * 5 +
                                               [f, ip, ip, vp, sz, vp, vp])
            lib.attn_fwd_paged_workspace_size.argtypes = [ip] * 8
            lib.attn_fwd_paged_workspace_size.restype = sz
            for fn in ("attn_page_table", "attn_cache_append", "attn_fwd_paged", "attn_rope",
                       "attn_cache_append_rope", "attn_cache_append_fp8", "attn_fwd_paged_fp8",
                       "attn_fwd", "attn_bwd", "attn_bwd_preprocess", "attn_bwd_main",
                       "attn_bwd_dq_convert", "attn_bwd_noalloc", "attn_fwd_varlen",
                       "attn_bwd_varlen"):
                getattr(lib, fn).restype = ctypes.c_int
            lib.attn_status_string.argtypes = [ctypes.c_int]
            lib.attn_status_string.restype = ctypes.c_char_p
            lib.attn_version.argtypes = []
            lib.attn_version.restype = ctypes.c_int
            _lib = lib
        return _lib


def attn_status_string(status: int) -> str:
    return library().attn_status_string(int(status)).decode()


def attn_version() -> int:
    return int(library().attn_version())


def attn_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(library().attn_bwd_workspace_size(B, H, N, d))


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _shape(q: torch.Tensor):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("expected a [B, H, N, d] tensor")
    _check_like("q", q, q)
    return tuple(int(x) for x in q.shape)


def _check_like(name: str, t: torch.Tensor, ref: torch.Tensor):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError(f"{name} must match q in shape, dtype and device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_gpu(q: torch.Tensor):
    """Every tensor argument has been checked to be on q's device; that device
    must be a CUDA one (a host pointer handed to a kernel would be read or
    written as if it were device memory)."""
    if not q.is_cuda:
        raise ValueError("the tensors must be on a CUDA device")


def _check_lse(lse, shape, q: torch.Tensor):
    """The log-sum-exp buffer: contiguous float32 of `shape` on q's device."""
    if (not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32
            or tuple(lse.shape) != tuple(shape) or lse.device != q.device
            or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {tuple(shape)} "
                         "on q's device")
    return lse


def _check_status(dev_status, q: torch.Tensor):
    """dev_status: None, or an int32 tensor (at least one element) on q's device."""
    if dev_status is None:
        return None
    if (not isinstance(dev_status, torch.Tensor) or dev_status.dtype != torch.int32
            or dev_status.numel() < 1 or dev_status.device != q.device
            or not dev_status.is_contiguous()):
        raise ValueError("dev_status must be a contiguous int32 tensor with at least one "
                         "element on q's device")
    return dev_status


def _check_workspace(workspace, q: torch.Tensor):
    if (not isinstance(workspace, torch.Tensor) or workspace.device != q.device
            or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on q's device")
    return workspace


def _keys(q: torch.Tensor, k: torch.Tensor) -> int:
    """Nk of k, which must be [B, H, Nk, d] like q apart from its length."""
    if (not isinstance(k, torch.Tensor) or k.dim() != 4 or k.shape[:2] != q.shape[:2]
            or k.shape[3] != q.shape[3] or k.dtype != q.dtype or k.device != q.device):
        raise ValueError("k must be [B, H, Nk, d] with q's B, H, d, dtype and device")
    if not k.is_contiguous():
        raise ValueError("k must be contiguous")
    return int(k.shape[2])


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DTYPE[t.dtype]


def _key_lens(key_lens, q):
    if key_lens is None:
        return None
    if (key_lens.dtype != torch.int32 or key_lens.device != q.device or key_lens.dim() != 1
            or key_lens.shape[0] != q.shape[0] or not key_lens.is_contiguous()):
        raise ValueError("key_lens must be a contiguous int32 [B] tensor on q's device")
    return key_lens


def _raise(st: int, where: str):
    if st != 0:
        raise AttnError(st, where)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def attn_fwd(q, k, v, *, causal: bool = False, window: int = 0, key_lens=None,
             dropout_p: float = 0.0,
             seed: int = 0, scale: Optional[float] = None, out=None, lse=None,
             dev_status=None, stream=None):
    """O, LSE = attention(q, k, v); see include/gbattn.h for the exact contract."""
    B, H, N, d = _shape(q)
    _check_like("q", q, q)
    Nk = _keys(q, k)
    _check_like("v", v, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q.shape, dtype=_out_dtype(q), device=q.device)
    if out.shape != q.shape or out.dtype != _out_dtype(q) or out.device != q.device \
            or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape (bf16 for e4m3 q)")
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_lse(lse, (B, H, N), q)
    _check_status(dev_status, q)
    kl = _key_lens(key_lens, q)
    _on_gpu(q)
    st = library().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, Nk, d,
                            _dtype_code(q), float(scale), int(bool(causal)), int(window), _ptr(kl),
                            float(dropout_p), int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(dev_status),
                            _stream(stream))
    _raise(st, "attn_fwd")
    return out, lse


def _workspace(B, H, N, d, workspace, q):
    need = attn_bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check_workspace(workspace, q)
    return workspace, int(workspace.numel() * workspace.element_size())


def attn_bwd(q, k, v, o, do, lse, *, causal: bool = False, window: int = 0, key_lens=None,
             dropout_p: float = 0.0, seed: int = 0, scale: Optional[float] = None, dq=None,
             dk=None, dv=None, workspace=None, dev_status=None, stream=None):
    """dQ, dK, dV of attention given the forward's o and lse and the gradient do."""
    B, H, N, d = _shape(q)
    Nk = _keys(q, k)
    for name, t in (("o", o), ("do", do)):
        _check_like(name, t, q)
    _check_like("v", v, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    _check_like("dq", dq, q)
    _check_like("dk", dk, k)
    _check_like("dv", dv, k)
    _check_lse(lse, (B, H, N), q)
    _check_status(dev_status, q)
    ws, ws_bytes = _workspace(B, H, N, d, workspace, q)
    kl = _key_lens(key_lens, q)
    _on_gpu(q)
    st = library().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                            _ptr(dk), _ptr(dv), B, H, N, Nk, d, _dtype_code(q), float(scale),
                            int(bool(causal)), int(window), _ptr(kl), float(dropout_p),
                            int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(ws), ws_bytes, _ptr(dev_status),
                            _stream(stream))
    _raise(st, "attn_bwd")
    return dq, dk, dv


def attn_bwd_noalloc(q, k, v, o, do, lse, *, causal: bool = False, window: int = 0,
                     key_lens=None,
                     dropout_p: float = 0.0, seed: int = 0, scale: Optional[float] = None,
                     dq=None, dk=None, dv=None, dev_status=None, stream=None):
    """attn_bwd using the library's built-in 32 MiB scratch instead of a
    workspace, for callers that cannot allocate device memory.  Outputs must be
    passed in (dq, dk, dv) by such callers; see include/gbattn.h."""
    B, H, N, d = _shape(q)
    Nk = _keys(q, k)
    for name, t in (("o", o), ("do", do)):
        _check_like(name, t, q)
    _check_like("v", v, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    _check_like("dq", dq, q)
    _check_like("dk", dk, k)
    _check_like("dv", dv, k)
    _check_lse(lse, (B, H, N), q)
    _check_status(dev_status, q)
    kl = _key_lens(key_lens, q)
    _on_gpu(q)
    st = library().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                    _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, Nk, d, _dtype_code(q),
                                    float(scale), int(bool(causal)), int(window), _ptr(kl),
                                    float(dropout_p),
                                    int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(dev_status),
                                    _stream(stream))
    _raise(st, "attn_bwd_noalloc")
    return dq, dk, dv


def attn_bwd_preprocess(o, do, lse, workspace, *, stream=None):
    B, H, N, d = _shape(o)
    _check_like("do", do, o)
    _check_lse(lse, (B, H, N), o)
    _check_workspace(workspace, o)
    _on_gpu(o)
    st = library().attn_bwd_preprocess(_ptr(o), _ptr(do), _ptr(lse), B, H, N, d,
                                       _dtype_code(o), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream))
    _raise(st, "attn_bwd_preprocess")


def attn_bwd_main(q, k, v, do, dk, dv, workspace, *, causal=False, window=0, key_lens=None,
                  dropout_p=0.0, seed=0, scale=None, dev_status=None, stream=None):
    B, H, N, d = _shape(q)
    Nk = _keys(q, k)
    _check_like("v", v, k)
    _check_like("do", do, q)
    _check_like("dk", dk, k)
    _check_like("dv", dv, k)
    _check_workspace(workspace, q)
    _check_status(dev_status, q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    kl = _key_lens(key_lens, q)
    _on_gpu(q)
    st = library().attn_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dk), _ptr(dv), B, H,
                                 N, Nk, d, _dtype_code(q), float(scale), int(bool(causal)),
                                 int(window), _ptr(kl),
                                 float(dropout_p), int(seed) & 0xFFFFFFFFFFFFFFFF,
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _ptr(dev_status), _stream(stream))
    _raise(st, "attn_bwd_main")


def attn_bwd_dq_convert(dq, workspace, *, scale=None, stream=None):
    B, H, N, d = _shape(dq)
    _check_workspace(workspace, dq)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _on_gpu(dq)
    st = library().attn_bwd_dq_convert(_ptr(dq), B, H, N, d, _dtype_code(dq), float(scale),
                                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream(stream))
    _raise(st, "attn_bwd_dq_convert")


# ---------------------------------------------------------------------------
# packed variable-length sequences
# ---------------------------------------------------------------------------
def _packed(name: str, t: torch.Tensor, H: int, d: int, ref: torch.Tensor):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if (t.dim() != 3 or t.shape[1] != H or t.shape[2] != d or t.dtype != ref.dtype
            or t.device != ref.device):
        raise ValueError(f"{name} must be [total, H, d] with q's H, d, dtype and device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return int(t.shape[0])


def _cu(name: str, cu, q: torch.Tensor) -> int:
    if (not isinstance(cu, torch.Tensor) or cu.dtype != torch.int32 or cu.device != q.device
            or cu.dim() != 1 or cu.numel() < 2 or not cu.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 [B + 1] tensor on q's device")
    return int(cu.numel()) - 1


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int, *,
                    causal: bool = False, window: int = 0, dropout_p: float = 0.0, seed: int = 0,
                    scale: Optional[float] = None, out=None, lse=None, dev_status=None,
                    stream=None):
    """Attention over packed sequences: q [total_q, H, d], k, v [total_k, H, d],
    sequence b at rows [cu[b], cu[b+1]).  Returns O [total_q, H, d] and LSE
    [H, total_q]; see include/gbattn.h."""
    if q.dim() != 3:
        raise ValueError("expected q as [total_q, H, d]")
    total_q, H, d = (int(x) for x in q.shape)
    _packed("q", q, H, d, q)
    total_k = _packed("k", k, H, d, q)
    if _packed("v", v, H, d, q) != total_k:
        raise ValueError("v must match k")
    B = _cu("cu_seqlens_q", cu_seqlens_q, q)
    if _cu("cu_seqlens_k", cu_seqlens_k, q) != B:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q.shape, dtype=_out_dtype(q), device=q.device)
    if out.shape != q.shape or out.dtype != _out_dtype(q) or out.device != q.device \
            or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape (bf16 for e4m3 q)")
    if lse is None:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    _check_lse(lse, (H, total_q), q)
    _check_status(dev_status, q)
    _on_gpu(q)
    st = library().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                   _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, H, total_q, total_k,
                                   int(max_seqlen_q), int(max_seqlen_k), d, _dtype_code(q),
                                   float(scale), int(bool(causal)), int(window), float(dropout_p),
                                   int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(dev_status),
                                   _stream(stream))
    _raise(st, "attn_fwd_varlen")
    return out, lse


def attn_bwd_varlen(q, k, v, o, do, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                    max_seqlen_k: int, *, causal: bool = False, window: int = 0,
                    dropout_p: float = 0.0, seed: int = 0, scale: Optional[float] = None,
                    dq=None, dk=None, dv=None, workspace=None, dev_status=None, stream=None):
    """dQ, dK, dV of attn_fwd_varlen (same packed layouts)."""
    if q.dim() != 3:
        raise ValueError("expected q as [total_q, H, d]")
    total_q, H, d = (int(x) for x in q.shape)
    _packed("q", q, H, d, q)
    total_k = _packed("k", k, H, d, q)
    if _packed("v", v, H, d, q) != total_k:
        raise ValueError("v must match k")
    for name, t in (("o", o), ("do", do)):
        _check_like(name, t, q)
    B = _cu("cu_seqlens_q", cu_seqlens_q, q)
    if _cu("cu_seqlens_k", cu_seqlens_k, q) != B:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    _check_like("dq", dq, q)
    _check_like("dk", dk, k)
    _check_like("dv", dv, k)
    _check_lse(lse, (H, total_q), q)
    _check_status(dev_status, q)
    ws, ws_bytes = _workspace(B, H, int(max_seqlen_q), d, workspace, q)
    _on_gpu(q)
    st = library().attn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                   _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q),
                                   _ptr(cu_seqlens_k), B, H, total_q, total_k, int(max_seqlen_q),
                                   int(max_seqlen_k), d, _dtype_code(q), float(scale),
                                   int(bool(causal)), int(window), float(dropout_p),
                                   int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(ws), ws_bytes,
                                   _ptr(dev_status), _stream(stream))
    _raise(st, "attn_bwd_varlen")
    return dq, dk, dv


# ---------------------------------------------------------------------------
# paged key/value cache
# ---------------------------------------------------------------------------
# The calls of a decoding step take a few microseconds on the GPU, so the host
# side is kept short.  The ordinary call (all arguments as documented, the
# current stream and device) is checked and marshalled by csrc/binding.cpp; what
# that does not take, refusals included, goes on here, with one pass over each
# tensor's attributes and plain integers for pointers and streams (a
# current_stream() object alone costs 3 us).
_native_module = None


def _native():
    """The extension lib/_binding.so.  Raises if it has not been built."""
    global _native_module
    if _native_module is None:
        lib = library()
        if not os.path.exists(_build.BINDING_PATH):
            raise RuntimeError(f"{_build.BINDING_PATH} is missing: build it with "
                               "exact_attention_58_gb300._build.build()")
        loader = importlib.machinery.ExtensionFileLoader("_binding", _build.BINDING_PATH)
        spec = importlib.util.spec_from_file_location("_binding", _build.BINDING_PATH, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value for fn in
                      ("attn_page_table", "attn_cache_append", "attn_fwd_paged",
                       "attn_fwd_paged_workspace_size", "attn_rope", "attn_cache_append_rope",
                       "attn_cache_append_fp8", "attn_fwd_paged_fp8")))
        _native_module = module
    return _native_module


def _int_tensor(name: str, t, dtype, shape, ref: torch.Tensor) -> int:
    """Pointer of a contiguous index tensor of the given type and shape on
    ref's device."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape
            or t.get_device() != ref.get_device() or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{ref.device}")
    return t.data_ptr()


def _cache_pair(k_cache, v_cache, d: int, ref: torch.Tensor, dtype=None):
    """Sizes and strides of the caches: [num_pages, Hkv, page_size, d] views of
    the given dtype (None: ref's) on ref's device, d innermost, laid out alike."""
    dtype = ref.dtype if dtype is None else dtype
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if (not isinstance(t, torch.Tensor) or t.dim() != 4 or t.dtype is not dtype
                or t.get_device() != ref.get_device()):
            raise ValueError(f"{name} must be [num_pages, Hkv, page_size, d], {dtype}, on "
                             f"{ref.device}")
    shape, strides = k_cache.shape, k_cache.stride()
    if shape[3] != d or strides[3] != 1:
        raise ValueError(f"the caches must have d = {d} innermost (stride 1)")
    if v_cache.shape != shape:
        raise ValueError("v_cache must match k_cache in shape")
    other = v_cache.stride()
    if other != strides and any(n > 1 and x != y for n, x, y in zip(shape, strides, other)):
        raise ValueError("v_cache must match k_cache in strides")
    return shape[0], shape[1], shape[2], strides[0], strides[1], strides[2]


def _rows(name: str, t):
    """Shape and strides of [tokens, heads, d] rows, d innermost, the other
    strides free."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [tokens, heads, d] tensor")
    strides = t.stride()
    if strides[2] != 1:
        raise ValueError(f"{name} must have d innermost (stride 1)")
    return t.shape, strides


def _new_rows(k, v):
    """Shape and strides of a step's k and v rows, which have to be laid out alike."""
    shape, strides = _rows("k", k)
    v_shape, v_strides = _rows("v", v)
    if (v_shape != shape or v.dtype is not k.dtype or v.get_device() != k.get_device()
            or (v_strides != strides
                and any(n > 1 and x != y for n, x, y in zip(shape, strides, v_strides)))):
        raise ValueError("v must match k in shape, strides, dtype and device")
    return shape, strides


def _call(fn, where: str, device: int, stream, *args):
    """fn(*args, stream) with `device` current: the library runs on the current
    device, and stream None is that device's current stream."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    elif isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    if device == torch._C._cuda_getDevice():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != 0:
        raise AttnError(st, where)


def _empty(shape, dtype, device: torch.device, stream):
    """An uninitialised tensor for work on `stream` (None: the current one).  It
    comes from that stream's memory, so nothing still running on another stream
    uses it, and what is freed after the call is handed out again behind it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _output(name: str, t, dtype, n: int, ref: torch.Tensor, stream):
    if t is None:
        return _empty(n, dtype, ref.device, stream)
    _int_tensor(name, t, dtype, (n,), ref)
    return t


def _int32(name: str, x) -> int:
    x = int(x)
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def attn_page_table(cached_lens, new_lens, page_table, free_pages, num_free, page_size: int,
                    max_tokens: int, *, cu_seqlens_q=None, seq_lens=None, slots=None,
                    pages_taken=None, dev_status=None, stream=None):
    """Page table and slot map of one serving step: request b has cached_lens[b]
    tokens in the cache and gets new_lens[b] more.  Enters the pages it needs
    into page_table ([B, max_pages], in place), taken from the end of
    free_pages[:num_free], and returns (cu_seqlens_q [B + 1], seq_lens [B],
    slots [max_tokens] int64, -1 behind the last token, pages_taken [1]).  All
    int32 CUDA tensors but slots; see include/gbattn.h."""
    if stream is None:
        done = (_native_module or _native()).page_table(
            cached_lens, new_lens, page_table, free_pages, num_free, page_size, max_tokens,
            cu_seqlens_q, seq_lens, slots, pages_taken, dev_status)
        if done is not None:
            return done
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [B, max_pages] tensor")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a one-dimensional int32 tensor")
    ref, i32 = page_table, torch.int32
    B, max_pages = ref.shape
    max_tokens = _int32("max_tokens", max_tokens)
    page_size = _int32("page_size", page_size)
    inputs = (_int_tensor("cached_lens", cached_lens, i32, (B,), ref),
              _int_tensor("new_lens", new_lens, i32, (B,), ref),
              _int_tensor("page_table", ref, i32, (B, max_pages), ref),
              _int_tensor("free_pages", free_pages, i32, free_pages.shape, ref),
              _int_tensor("num_free", num_free, i32, (1,), ref))
    _check_status(dev_status, ref)
    _on_gpu(ref)
    dev = ref.device

    cu_seqlens_q = _output("cu_seqlens_q", cu_seqlens_q, i32, B + 1, ref, stream)
    seq_lens = _output("seq_lens", seq_lens, i32, B, ref, stream)
    pages_taken = _output("pages_taken", pages_taken, i32, 1, ref, stream)
    slots = _output("slots", slots, torch.int64, max(max_tokens, 0), ref, stream)
    _call(library().attn_page_table, "attn_page_table", dev.index, stream, *inputs,
          cu_seqlens_q.data_ptr(), seq_lens.data_ptr(), slots.data_ptr(), pages_taken.data_ptr(),
          B, max_pages, page_size, max_tokens, free_pages.shape[0], _ptr(dev_status))
    return cu_seqlens_q, seq_lens, slots, pages_taken


def attn_cache_append(k, v, k_cache, v_cache, slots, *, dev_status=None, stream=None):
    """Writes k, v ([T, Hkv, d], d innermost, the same strides) into slots
    slots[t] (int64 [T]; -1 skips a token) of the caches ([num_pages, Hkv,
    page_size, d] views of like strides); see include/gbattn.h."""
    if stream is None and (_native_module or _native()).cache_append(k, v, k_cache, v_cache, slots,
                                                                     dev_status):
        return
    (T, Hkv, d), strides = _new_rows(k, v)
    pages, heads, page_size, sp, sh, st = _cache_pair(k_cache, v_cache, d, k)
    if heads != Hkv:
        raise ValueError("the caches must have k's number of heads")
    at = _int_tensor("slots", slots, torch.int64, (T,), k)
    _check_status(dev_status, k)
    _on_gpu(k)
    _call(library().attn_cache_append, "attn_cache_append", k.get_device(), stream, k.data_ptr(),
          v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), at, T, Hkv, d, _dtype_code(k),
          strides[0], strides[1], pages, page_size, sp, sh, st, _ptr(dev_status))


def attn_fwd_paged_workspace_size(B: int, H: int, Hkv: int, total_q: int, max_seqlen_q: int,
                                  max_pages: int, page_size: int, d: int) -> int:
    return int(library().attn_fwd_paged_workspace_size(B, H, Hkv, total_q, max_seqlen_q, max_pages,
                                                       page_size, d))


def attn_fwd_paged(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens_q, max_seqlen_q: int, *,
                   causal: bool = False, window: int = 0, scale: Optional[float] = None, out=None,
                   lse=None, workspace=None, dev_status=None, stream=None):
    """Attention of packed new tokens over a paged cache: q [total_q, H, d] (d
    innermost, other strides free), request b's queries at rows
    [cu_seqlens_q[b], cu_seqlens_q[b + 1]), the last of its seq_lens[b] key
    positions; keys and values in the pages that page_table [B, max_pages]
    names.  Query head h reads key head h // (H // Hkv).  Returns O [total_q,
    H, d] and LSE [H, total_q]; see include/gbattn.h."""
    if stream is None:
        done = (_native_module or _native()).fwd_paged(q, k_cache, v_cache, page_table, seq_lens,
                                                       cu_seqlens_q, max_seqlen_q, causal, window,
                                                       scale, out, lse, workspace, dev_status)
        if done is not None:
            return done
    return _fwd_paged("attn_fwd_paged", q, k_cache, v_cache, None, page_table, seq_lens,
                      cu_seqlens_q, max_seqlen_q, causal, window, scale, out, lse, workspace,
                      dev_status, stream)


def _fwd_paged(where, q, k_cache, v_cache, scales, page_table, seq_lens, cu_seqlens_q, max_seqlen_q,
               causal, window, scale, out, lse, workspace, dev_status, stream):
    """attn_fwd_paged, or with the scales of a cache of e4m3 attn_fwd_paged_fp8."""
    (total_q, H, d), strides = _rows("q", q)
    pages, Hkv, page_size, sp, sh, st = _cache_pair(
        k_cache, v_cache, d, q, None if scales is None else torch.float8_e4m3fn)
    scale_ptrs = () if scales is None else _scale_pair(*scales, pages, Hkv, q)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [B, max_pages] tensor")
    B, max_pages = page_table.shape
    table = _int_tensor("page_table", page_table, torch.int32, (B, max_pages), q)
    lens = _int_tensor("seq_lens", seq_lens, torch.int32, (B,), q)
    cu = _int_tensor("cu_seqlens_q", cu_seqlens_q, torch.int32, (B + 1,), q)
    _check_status(dev_status, q)
    max_seqlen_q = _int32("max_seqlen_q", max_seqlen_q)
    window = _int32("window", window)
    _on_gpu(q)
    dev = q.device
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((total_q, H, d), q.dtype, dev, stream)
    elif (not isinstance(out, torch.Tensor) or out.shape != q.shape or out.dtype is not q.dtype
          or out.get_device() != dev.index or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    if lse is None:
        lse = _empty((H, total_q), torch.float32, dev, stream)
    else:
        _check_lse(lse, (H, total_q), q)
    lib = library()
    ws_bytes = 0
    if workspace is None:
        ws_bytes = lib.attn_fwd_paged_workspace_size(B, H, Hkv, total_q, max_seqlen_q, max_pages,
                                                     page_size, d)
        if ws_bytes:
            workspace = _empty(ws_bytes, torch.uint8, dev, stream)
    else:
        _check_workspace(workspace, q)
        ws_bytes = workspace.numel() * workspace.element_size()
    _call(getattr(lib, where), where, dev.index, stream, q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), *scale_ptrs, out.data_ptr(), lse.data_ptr(), cu, lens, table, B, H, Hkv,
          total_q, max_seqlen_q, pages, page_size, max_pages, d, _dtype_code(q), strides[0], strides[1], sp,
          sh, st, float(scale), int(bool(causal)), window, _ptr(workspace), ws_bytes,
          _ptr(dev_status))
    return out, lse


def _scale_pair(k_scale, v_scale, pages: int, Hkv: int, ref: torch.Tensor):
    """Pointers of the scales of a cache of e4m3."""
    return tuple(_int_tensor(name, t, torch.float32, (pages, Hkv), ref)
                 for name, t in (("k_scale", k_scale), ("v_scale", v_scale)))


def attn_fwd_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_seqlens_q,
                       max_seqlen_q: int, *, causal: bool = False, window: int = 0,
                       scale: Optional[float] = None, out=None, lse=None, workspace=None,
                       dev_status=None, stream=None):
    """attn_fwd_paged over a cache of 8 bits: torch.float8_e4m3fn caches, whose
    page and head stand for their values times k_scale and v_scale (float32 [num_pages,
    Hkv], powers of two).  q and O are bf16 or fp16; see include/gbattn.h."""
    if stream is None:
        done = (_native_module or _native()).fwd_paged_fp8(
            q, k_cache, v_cache, page_table, seq_lens, cu_seqlens_q, max_seqlen_q, causal, window,
            scale, out, lse, workspace, dev_status, k_scale, v_scale)
        if done is not None:
            return done
    return _fwd_paged("attn_fwd_paged_fp8", q, k_cache, v_cache, (k_scale, v_scale), page_table,
                      seq_lens, cu_seqlens_q, max_seqlen_q, causal, window, scale, out, lse,
                      workspace, dev_status, stream)


def attn_cache_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, slots, *, dev_status=None,
                          stream=None):
    """attn_cache_append into a cache of 8 bits (see attn_fwd_paged_fp8): each
    page and head gets the smallest scale that holds its rows, and rows that it held
    before are rounded again where that grows; see include/gbattn.h."""
    if stream is None and (_native_module or _native()).cache_append_fp8(
            k, v, k_cache, v_cache, slots, dev_status, k_scale, v_scale):
        return
    (T, Hkv, d), strides = _new_rows(k, v)
    pages, heads, page_size, sp, sh, st = _cache_pair(k_cache, v_cache, d, k, torch.float8_e4m3fn)
    if heads != Hkv:
        raise ValueError("the caches must have k's number of heads")
    scales = _scale_pair(k_scale, v_scale, pages, Hkv, k)
    at = _int_tensor("slots", slots, torch.int64, (T,), k)
    _check_status(dev_status, k)
    _on_gpu(k)
    _call(library().attn_cache_append_fp8, "attn_cache_append_fp8", k.get_device(), stream,
          k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), *scales, at, T, Hkv, d,
          _dtype_code(k), strides[0], strides[1], pages, page_size, sp, sh, st, _ptr(dev_status))


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def attn_rope_frequencies(rotary_dim: int, base: float = 10000.0, *, factor: float = 1.0,
                          method: str = "linear", original_len: int = 0, fast: float = 32.0,
                          slow: float = 1.0, device=None):
    """(inv_freq, scaling) for attn_rope: float32 [rotary_dim / 2] and a number.
    Frequencies base^(-2i / rotary_dim); for contexts `factor` times as long as
    the original_len positions that a model was trained on they are
      "linear"  divided by factor (positions interpolated);
      "base"    those of the base times factor^(rotary_dim / (rotary_dim - 2)): the
                highest stays, the lowest is divided by factor;
      "parts"   kept where original_len positions make `fast` turns or more, divided
                by factor where they make `slow` or fewer, and in between mixed
                linearly over i; cosines and sines times 0.1 ln(factor) + 1."""
    if rotary_dim < 2 or rotary_dim % 2 != 0:
        raise ValueError("rotary_dim must be even and positive")
    if not (base > 1.0 and math.isfinite(base) and factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor at least 1")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    scaling = 1.0
    if method == "base":
        if rotary_dim < 4:
            raise ValueError("the base method needs two frequencies")
        base *= factor ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-i / rotary_dim)
    if method == "linear":
        freq = freq / factor
    elif method == "parts":
        if original_len < 1 or not fast > slow > 0.0:
            raise ValueError("the parts method needs original_len and fast > slow > 0")
        # index whose frequency makes `turns` turns in original_len positions
        def index(turns):
            return rotary_dim * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = math.floor(index(fast)), math.ceil(index(slow))
        mix = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        freq = freq * (1.0 - mix) + freq / factor * mix
        scaling = 0.1 * math.log(factor) + 1.0
    elif method != "base":
        raise ValueError(f"unknown method {method!r}")
    return freq.float().to(device), scaling


def _rope_rows(name: str, t, ref: torch.Tensor):
    """(B, heads, N, d) and the strides of batch, head and token of [B, heads, N,
    d] or packed [tokens, heads, d] rows, d innermost."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (3, 4) or t.dim() != ref.dim():
        raise ValueError(f"{name} must be [B, heads, N, d] or [tokens, heads, d], as q")
    if t.dtype is not ref.dtype or t.get_device() != ref.get_device():
        raise ValueError(f"{name} must match q in dtype and device")
    n, s = t.shape, t.stride()
    if s[-1] != 1:
        raise ValueError(f"{name} must have d innermost (stride 1)")
    if t.dim() == 3:
        return (1, n[1], n[0], n[2]), (0, s[1], s[0])
    return tuple(n), s[:3]


def _rope_out(name: str, out, like: torch.Tensor, stream):
    """The output given, or None's new tensor, and its strides."""
    if out is None:
        _on_gpu(like)
        out = _empty(tuple(like.shape), like.dtype, like.device, stream)
    elif not isinstance(out, torch.Tensor) or out.shape != like.shape:
        raise ValueError(f"{name} must have its input's shape")
    return out, _rope_rows(name, out, like)[1]


def _inv_freq(t, ref: torch.Tensor):
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError("inv_freq must be a float32 [rotary_dim / 2] tensor")
    return _int_tensor("inv_freq", t, torch.float32, t.shape, ref), 2 * t.shape[0]


def attn_rope(q, k, inv_freq, positions=None, *, interleaved: bool = False, inverse: bool = False,
              scaling: float = 1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions: q [B, H, N, d] and k [B, Hk, N, d] (or packed [T, H, d] and
    [T, Hk, d]; k may be None), d innermost, other strides free.  inv_freq: float32
    [rotary_dim / 2]; positions: int32 [N], [B, N] or, packed, [T]; None: 0 .. N - 1
    (not for packed rows).  inverse=True is the transposed map: gradients of q and k from those of
    the results.  Returns (q_out, k_out); q_out=q works in place.  See include/gbattn.h."""
    if stream is None:
        done = (_native_module or _native()).rope(q, k, inv_freq, positions, interleaved, inverse,
                                                  scaling, q_out, k_out)
        if done is not None:
            return done
    if not isinstance(q, torch.Tensor):
        raise ValueError("q must be a tensor")
    (B, H, N, d), qs = _rope_rows("q", q, q)
    freq, rotary_dim = _inv_freq(inv_freq, q)
    Hk, ks = 0, (0, 0, 0)
    if k is not None:
        (kB, Hk, kN, kd), ks = _rope_rows("k", k, q)
        if (kB, kN, kd) != (B, N, d):
            raise ValueError("k must match q in all but the number of heads")
        if Hk < 1:
            raise ValueError("k has no heads")
    elif k_out is not None:
        raise ValueError("k_out needs k")
    pos, pos_batch = None, 0
    if positions is not None:
        rows = q.dim() == 4 and isinstance(positions, torch.Tensor) and positions.dim() == 2
        pos = _int_tensor("positions", positions, torch.int32, (B, N) if rows else (N,), q)
        pos_batch = N if rows else 0
    elif q.dim() == 3:
        raise ValueError("packed rows need positions")
    q_out, qo = _rope_out("q_out", q_out, q, stream)
    ko = (0, 0, 0)
    if k is not None:
        k_out, ko = _rope_out("k_out", k_out, k, stream)
    _on_gpu(q)
    _call(library().attn_rope, "attn_rope", q.get_device(), stream, q.data_ptr(),
          None if k is None else k.data_ptr(), q_out.data_ptr(),
          None if k is None else k_out.data_ptr(), freq, pos, B, H, Hk, N, d, rotary_dim,
          _dtype_code(q), *qs, *ks, *qo, *ko, pos_batch, float(scaling), int(bool(interleaved)),
          int(bool(inverse)))
    return q_out, (None if k is None else k_out)


def attn_cache_append_rope(q, k, v, k_cache, v_cache, slots, inv_freq, positions=None, *,
                           cu_seqlens_q=None, seq_lens=None, interleaved: bool = False,
                           scaling: float = 1.0, q_out=None, dev_status=None, stream=None):
    """attn_cache_append with rotary positions on the way: the rotated k ([T, Hkv, d])
    and v go into the caches, and the rotated q ([T, H, d]) is returned (q_out=q works
    in place).  positions: int32 [T], or cu_seqlens_q and seq_lens as attn_page_table
    gives them.  See include/gbattn.h."""
    if stream is None:
        done = (_native_module or _native()).cache_append_rope(
            q, k, v, k_cache, v_cache, slots, inv_freq, positions, cu_seqlens_q, seq_lens,
            interleaved, scaling, q_out, dev_status)
        if done is not None:
            return done
    (T, Hkv, d), strides = _new_rows(k, v)
    (q_T, H, q_d), qs = _rows("q", q)
    if q_T != T or q_d != d or q.dtype is not k.dtype or q.get_device() != k.get_device():
        raise ValueError("q must match k in all but the number of heads")
    pages, heads, page_size, sp, sh, st = _cache_pair(k_cache, v_cache, d, k)
    if heads != Hkv:
        raise ValueError("the caches must have k's number of heads")
    at = _int_tensor("slots", slots, torch.int64, (T,), k)
    freq, rotary_dim = _inv_freq(inv_freq, k)
    pos = cu = lens = None
    B = 0
    if positions is not None:
        pos = _int_tensor("positions", positions, torch.int32, (T,), k)
    else:
        if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
            raise ValueError("positions, or cu_seqlens_q and seq_lens, are needed")
        B = seq_lens.shape[0]
        lens = _int_tensor("seq_lens", seq_lens, torch.int32, (B,), k)
        cu = _int_tensor("cu_seqlens_q", cu_seqlens_q, torch.int32, (B + 1,), k)
    _check_status(dev_status, k)
    q_out, qo = _rope_out("q_out", q_out, q, stream)
    _on_gpu(k)
    _call(library().attn_cache_append_rope, "attn_cache_append_rope", k.get_device(), stream,
          q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), at, freq, pos, cu, lens, B, T, H, Hkv, d, rotary_dim, _dtype_code(k),
          qs[0], qs[1], strides[0], strides[1], qo[2], qo[1], pages, page_size, sp, sh, st,
          float(scaling), int(bool(interleaved)), _ptr(dev_status))
    return q_out


def attn_selftest_wait(dev_status, *, arrive: bool, stream=None):
    """Device self-test of the bounded waits (see include/gbattn.h): with
    arrive=False the wait expires and ATTN_ERR_DEVICE_TIMEOUT lands in
    dev_status (a CUDA int32 tensor, 0 on entry)."""
    st = library().attn_selftest_wait(_ptr(dev_status), int(bool(arrive)), _stream(stream))
    _raise(st, "attn_selftest_wait")


def attn_selftest_fwd_withheld(q, k, v, dev_status, *, withhold_block: int, wait_ms: int = 20,
                               out=None, lse=None, stream=None):
    """Device self-test of the forward kernel's abort path (see
    include/gbattn.h): bf16 [B, H, N, 128] q and [B, H, Nk, 128] k, v; the K
    tile of key block `withhold_block` is never loaded (< 0: nothing withheld)
    and waits give up after `wait_ms`.  dev_status: a CUDA int32 tensor, 0 on
    entry."""
    B, H, N, d = _shape(q)
    Nk = _keys(q, k)
    _check_like("v", v, k)
    if q.dtype != torch.bfloat16 or d != 128:
        raise ValueError("the self test runs bf16 with d = 128")
    out = torch.empty_like(q) if out is None else out
    _check_like("out", out, q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check_lse(lse, (B, H, N), q)
    if _check_status(dev_status, q) is None:
        raise ValueError("dev_status is required")
    _on_gpu(q)
    st = library().attn_selftest_fwd_withheld(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B,
                                              H, N, Nk, int(withhold_block), int(wait_ms),
                                              _ptr(dev_status), _stream(stream))
    _raise(st, "attn_selftest_fwd_withheld")
    return out, lse
