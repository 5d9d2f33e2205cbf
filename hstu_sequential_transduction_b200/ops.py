"""Python binding of libhstu (ctypes): argument marshalling only.

Every function here has the name of the C entry point it calls (include/hstu.h)
and does no arithmetic of the method: it checks tensor placement, allocates
outputs and workspace through PyTorch's allocator, and passes raw device
pointers plus the current CUDA stream.  There is no fallback: if the library
cannot be loaded or built, every call raises.
"""

from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional

import torch

from . import build as _build

HSTU_F32, HSTU_BF16 = 0, 1
# hstu_attn_desc.debug_checks: the bounded-wait test hooks (see include/hstu.h)
HSTU_DEBUG_WAIT_TEST = 2
HSTU_DEBUG_CACHE_WAIT_TEST = 4
STATUS = {0: "HSTU_OK", 1: "HSTU_ERR_INVALID_ARG", 2: "HSTU_ERR_UNSUPPORTED", 3: "HSTU_ERR_WORKSPACE",
          4: "HSTU_ERR_CUDA", 5: "HSTU_ERR_DEVICE_CHECK"}

EXPORTED = ["hstu_status_string", "hstu_version", "hstu_attn_workspace_size",
            "hstu_layer_workspace_size", "hstu_attn_fwd", "hstu_attn_bwd", "hstu_layer_fwd",
            "hstu_check_device_flag", "hstu_debug_bias_indices", "hstu_debug_schedule",
            "hstu_attn_fwd_noalloc", "hstu_layer_bwd_workspace_size", "hstu_layer_bwd",
            "hstu_jagged_truncate", "hstu_quantize_weight_e4m3", "hstu_quantize_rows_e4m3", "hstu_gemm_e4m3",
            "hstu_e4m3_weight_bytes", "hstu_cache_append_workspace_size", "hstu_cache_append",
            "hstu_cache_attn_workspace_size", "hstu_cache_attn_fwd", "hstu_cache_evict_workspace_size",
            "hstu_cache_evict"]
# tokens of a page of the 8-bit key/value cache
HSTU_CACHE_PAGE = 64


class HstuError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class hstu_attn_desc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("total_tokens", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("inv_n", ctypes.c_float), ("pos_lo", ctypes.c_int32), ("pos_hi", ctypes.c_int32),
                ("num_time_buckets", ctypes.c_int32), ("debug_checks", ctypes.c_int32),
                ("local_window", ctypes.c_int32), ("global_window", ctypes.c_int32), ("fp8_qk", ctypes.c_int32),
                ("cand_positions", ctypes.c_int32), ("per_head_tables", ctypes.c_int32)]


class hstu_layer_desc(ctypes.Structure):
    _fields_ = [("attn", hstu_attn_desc), ("d_model", ctypes.c_int32), ("ln_eps", ctypes.c_float),
                ("output_concat", ctypes.c_int32), ("fp8_projections", ctypes.c_int32)]


class hstu_cache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("timestamps", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("weights", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load_library(allow_build: bool = True) -> ctypes.CDLL:
    """Load libhstu.so, compiling it first when it is missing or stale."""
    global _lib
    with _lock:
        if _lib is None:
            if allow_build and _build.needs_build():
                _build.build()
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"libhstu.so not found at {_build.LIB}; build it with "
                                   "python -m hstu_sequential_transduction_b200.build")
            lib = ctypes.CDLL(_build.LIB)
            lib.hstu_status_string.restype = ctypes.c_char_p
            lib.hstu_status_string.argtypes = [ctypes.c_int]
            lib.hstu_version.restype = ctypes.c_int
            for name in EXPORTED[2:]:
                getattr(lib, name).restype = ctypes.c_int
            # the cache's calls come once per token: with argument types they take plain integers
            p, i, n, z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            lib.hstu_cache_append.argtypes = [p, i, i, i, n, p, n, p, n] + [p] * 9 + [z, p]
            lib.hstu_cache_attn_workspace_size.argtypes = [p, p, i, i, p]
            lib.hstu_cache_attn_fwd.argtypes = [p, p, i, p, n] + [p] * 12 + [z, p]
            lib.hstu_cache_evict_workspace_size.argtypes = [p, i, i, i, p]
            lib.hstu_cache_evict.argtypes = [p] + [i] * 5 + [p] * 7 + [z, p]
            lib.hstu_e4m3_weight_bytes.restype = ctypes.c_size_t
            lib.hstu_e4m3_weight_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32]
            _lib = lib
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn: str, status: int):
    if status != 0:
        raise HstuError(fn, status)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return HSTU_BF16
    if t.dtype == torch.float32:
        return HSTU_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dev(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def make_attn_desc(num_seqs, max_seq_len, total_tokens, num_heads, d_qk, d_v, dtype, inv_n,
                   pos_lo, pos_hi, num_time_buckets, local_window=0, global_window=0,
                   fp8_qk=False, cand_own_index=False, per_head_tables=False) -> hstu_attn_desc:
    return hstu_attn_desc(int(num_seqs), int(max_seq_len), int(total_tokens), int(num_heads),
                          int(d_qk), int(d_v), int(dtype), float(inv_n), int(pos_lo), int(pos_hi),
                          int(num_time_buckets), 0, int(local_window), int(global_window), int(bool(fp8_qk)),
                          int(bool(cand_own_index)), int(bool(per_head_tables)))


def hstu_status_string(status: int) -> str:
    return load_library().hstu_status_string(int(status)).decode()


def hstu_version() -> int:
    return load_library().hstu_version()


def hstu_attn_workspace_size(desc: hstu_attn_desc, is_bwd: bool) -> int:
    n = ctypes.c_size_t(0)
    _check("hstu_attn_workspace_size",
           load_library().hstu_attn_workspace_size(ctypes.byref(desc), int(is_bwd), ctypes.byref(n)))
    return n.value


def hstu_layer_workspace_size(desc: hstu_layer_desc) -> int:
    n = ctypes.c_size_t(0)
    _check("hstu_layer_workspace_size",
           load_library().hstu_layer_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _tables(rab_pos, rab_time, num_heads, pos_lo, pos_hi):
    """(num_time_buckets, per_head) of a pair of bias tables: both 1-D (shared by
    the heads) or both [num_heads, n] (one row per head)."""
    npos = int(pos_hi) - int(pos_lo) + 1
    if rab_pos.dim() != rab_time.dim() or rab_pos.dim() not in (1, 2):
        raise ValueError("rab_pos and rab_time must both be 1-D or both [num_heads, n]")
    per_head = rab_pos.dim() == 2
    if per_head and (rab_pos.shape[0] != num_heads or rab_time.shape[0] != num_heads):
        raise ValueError(f"per-head tables need {num_heads} rows")
    if rab_pos.shape[-1] != npos:
        raise ValueError(f"rab_pos has {rab_pos.shape[-1]} entries for distances {pos_lo}..{pos_hi}")
    return rab_time.shape[-1], per_head


def _attn_desc_from(q, v, seq_offsets, max_seq_len, inv_n, pos_lo, pos_hi, rab_pos, rab_time, local_window=0,
                    global_window=0, fp8_qk=False, cand_own_index=False):
    nb, per_head = _tables(rab_pos, rab_time, q.shape[1], pos_lo, pos_hi)
    return make_attn_desc(seq_offsets.numel() - 1, max_seq_len, q.shape[0], q.shape[1], q.shape[2],
                          v.shape[2], _dtype_code(q), inv_n, pos_lo, pos_hi, nb, local_window,
                          global_window, fp8_qk, cand_own_index, per_head)


def hstu_attn_fwd(q, k, v, seq_offsets, timestamps, num_targets, rab_pos, rab_time, *,
                  max_seq_len: int, inv_n: float, pos_lo: int, pos_hi: int, out=None,
                  workspace=None, stream=None, local_window: int = 0, global_window: int = 0,
                  fp8_qk: bool = False, cand_own_index: bool = False):
    """O = jagged SiLU attention; q, k [T, H, d_qk], v [T, H, d_v] on CUDA.
    local_window > 0 applies the semi-local mask; fp8_qk computes Q K^T on E4M3
    codes of q and k; cand_own_index puts candidate i at position i; 2-D tables
    [H, n] give each head its own (see hstu_attn_desc)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    _dev(seq_offsets, "seq_offsets", torch.int64)
    _dev(timestamps, "timestamps", torch.int64)
    _dev(num_targets, "num_targets", torch.int32)
    _dev(rab_pos, "rab_pos", torch.float32)
    _dev(rab_time, "rab_time", torch.float32)
    desc = _attn_desc_from(q, v, seq_offsets, max_seq_len, inv_n, pos_lo, pos_hi, rab_pos, rab_time, local_window,
                           global_window, fp8_qk, cand_own_index)
    if out is None:
        out = torch.empty_like(v)
    _dev(out, "out", q.dtype)
    need = hstu_attn_workspace_size(desc, False)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    _check("hstu_attn_fwd", load_library().hstu_attn_fwd(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets), _ptr(timestamps),
        _ptr(num_targets), _ptr(rab_pos), _ptr(rab_time), _ptr(out), _ptr(workspace),
        ctypes.c_size_t(workspace.numel()), _stream(stream)))
    return out


def hstu_attn_fwd_noalloc(q, k, v, seq_offsets, timestamps, num_targets, rab_pos, rab_time, out,
                          *, max_seq_len: int, inv_n: float, pos_lo: int, pos_hi: int, stream=None,
                          cand_own_index: bool = False):
    """hstu_attn_fwd without a workspace: the library keeps the scheduler's
    scratch in a static device array (for callers that cannot allocate).
    `out` must be preallocated; nothing is allocated here either."""
    desc = _attn_desc_from(q, v, seq_offsets, max_seq_len, inv_n, pos_lo, pos_hi, rab_pos, rab_time,
                           cand_own_index=cand_own_index)
    _check("hstu_attn_fwd_noalloc", load_library().hstu_attn_fwd_noalloc(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets), _ptr(timestamps),
        _ptr(num_targets), _ptr(rab_pos), _ptr(rab_time), _ptr(out), _stream(stream)))
    return out


def hstu_attn_bwd(q, k, v, seq_offsets, timestamps, num_targets, rab_pos, rab_time, dout, *,
                  max_seq_len: int, inv_n: float, pos_lo: int, pos_hi: int, grads=None,
                  workspace=None, stream=None, local_window: int = 0, global_window: int = 0,
                  cand_own_index: bool = False):
    """(dq, dk, dv, d_rab_pos, d_rab_time) for the loss sum(O * dout); the table
    gradients have the tables' shapes."""
    for name, t in (("q", q), ("k", k), ("v", v), ("dout", dout)):
        _dev(t, name, q.dtype)
    _dev(seq_offsets, "seq_offsets", torch.int64)
    _dev(timestamps, "timestamps", torch.int64)
    _dev(num_targets, "num_targets", torch.int32)
    desc = _attn_desc_from(q, v, seq_offsets, max_seq_len, inv_n, pos_lo, pos_hi, rab_pos, rab_time, local_window,
                           global_window, cand_own_index=cand_own_index)
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(rab_pos), torch.empty_like(rab_time))
    dq, dk, dv, drp, drt = grads
    need = hstu_attn_workspace_size(desc, True)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    _check("hstu_attn_bwd", load_library().hstu_attn_bwd(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets), _ptr(timestamps),
        _ptr(num_targets), _ptr(rab_pos), _ptr(rab_time), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
        _ptr(drp), _ptr(drt), _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream(stream)))
    return dq, dk, dv, drp, drt


def hstu_layer_fwd(x, w1, b1, w2, b2, ln_gamma, ln_beta, seq_offsets, timestamps, num_targets,
                   rab_pos, rab_time, *, num_heads: int, d_qk: int, d_v: int, max_seq_len: int,
                   inv_n: float, pos_lo: int, pos_hi: int, ln_eps: float = 1e-5, y=None,
                   saved_uvqk=None, saved_o=None, workspace=None, stream=None, output_concat: bool = False,
                   fp8_projections: bool = False, local_window: int = 0, global_window: int = 0,
                   cand_own_index: bool = False):
    """Y = f2(LayerNorm(attention(SiLU(f1(X)))) * U) for one layer; with
    output_concat, f2 reads [U | O | G] and w2 is [3 H d_v, D]; with
    fp8_projections, w1 and w2 are E4M3 weight packs (quantize_weight_e4m3)."""
    for name, t in (("x", x), ("b1", b1), ("b2", b2)) + (() if fp8_projections else (("w1", w1), ("w2", w2))):
        _dev(t, name, x.dtype)
    if fp8_projections:
        _dev(w1, "w1", torch.uint8)
        _dev(w2, "w2", torch.uint8)
    _dev(ln_gamma, "ln_gamma", torch.float32)
    _dev(ln_beta, "ln_beta", torch.float32)
    T, D = x.shape
    nb, per_head = _tables(rab_pos, rab_time, num_heads, pos_lo, pos_hi)
    attn = make_attn_desc(seq_offsets.numel() - 1, max_seq_len, T, num_heads, d_qk, d_v,
                          _dtype_code(x), inv_n, pos_lo, pos_hi, nb, local_window, global_window,
                          False, cand_own_index, per_head)
    desc = hstu_layer_desc(attn, int(D), float(ln_eps), int(bool(output_concat)), int(bool(fp8_projections)))
    if fp8_projections:
        W = num_heads * (2 * d_v + 2 * d_qk)
        for name, t, k, n in (("w1", w1, D, W), ("w2", w2, num_heads * d_v, D)):
            if t.numel() < hstu_e4m3_weight_bytes(k, n):
                raise ValueError(f"{name} is not an E4M3 pack of a [{k}, {n}] weight")
    elif w2.shape[0] != (3 if output_concat else 1) * num_heads * d_v:
        raise ValueError(f"w2 has {w2.shape[0]} rows for output_concat={output_concat}")
    if y is None:
        y = torch.empty((T, D), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(hstu_layer_workspace_size(desc), x.device)
    _check("hstu_layer_fwd", load_library().hstu_layer_fwd(
        ctypes.byref(desc), _ptr(x), _ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2), _ptr(ln_gamma),
        _ptr(ln_beta), _ptr(seq_offsets), _ptr(timestamps), _ptr(num_targets), _ptr(rab_pos),
        _ptr(rab_time), _ptr(y), _ptr(saved_uvqk), _ptr(saved_o), _ptr(workspace),
        ctypes.c_size_t(workspace.numel()), _stream(stream)))
    return y


def hstu_layer_bwd_workspace_size(desc: hstu_layer_desc) -> int:
    n = ctypes.c_size_t(0)
    _check("hstu_layer_bwd_workspace_size",
           load_library().hstu_layer_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def hstu_layer_bwd(x, w1, b1, w2, ln_gamma, ln_beta, seq_offsets, timestamps, num_targets, rab_pos, rab_time,
                   saved_uvqk, saved_o, dy, *, num_heads: int, d_qk: int, d_v: int, max_seq_len: int,
                   inv_n: float, pos_lo: int, pos_hi: int, ln_eps: float = 1e-5, workspace=None, stream=None,
                   output_concat: bool = False, local_window: int = 0, global_window: int = 0,
                   cand_own_index: bool = False):
    """Gradients of sum(Y * dy) for one layer (bf16): a dict with dx (bf16) and the
    float32 parameter gradients dw1, db1, dw2, db2, d_ln_gamma, d_ln_beta,
    d_rab_pos, d_rab_time (the tables' shapes; output_concat as in hstu_layer_fwd)."""
    for name, t in (("x", x), ("w1", w1), ("b1", b1), ("w2", w2), ("saved_uvqk", saved_uvqk),
                    ("saved_o", saved_o), ("dy", dy)):
        _dev(t, name, x.dtype)
    _dev(ln_gamma, "ln_gamma", torch.float32)
    _dev(ln_beta, "ln_beta", torch.float32)
    T, D = x.shape
    W = w1.shape[1]
    hv = num_heads * d_v
    nb, per_head = _tables(rab_pos, rab_time, num_heads, pos_lo, pos_hi)
    attn = make_attn_desc(seq_offsets.numel() - 1, max_seq_len, T, num_heads, d_qk, d_v,
                          _dtype_code(x), inv_n, pos_lo, pos_hi, nb, local_window, global_window,
                          False, cand_own_index, per_head)
    desc = hstu_layer_desc(attn, int(D), float(ln_eps), int(bool(output_concat)))
    F = (3 if output_concat else 1) * hv
    if w2.shape[0] != F:
        raise ValueError(f"w2 has {w2.shape[0]} rows for output_concat={output_concat}")
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"dx": torch.empty((T, D), dtype=x.dtype, device=dev), "dw1": torch.empty((D, W), **f32),
           "db1": torch.empty(W, **f32), "dw2": torch.empty((F, D), **f32), "db2": torch.empty(D, **f32),
           "d_ln_gamma": torch.empty(hv, **f32), "d_ln_beta": torch.empty(hv, **f32),
           "d_rab_pos": torch.empty(rab_pos.shape, **f32), "d_rab_time": torch.empty(rab_time.shape, **f32)}
    if workspace is None:
        workspace = alloc_workspace(hstu_layer_bwd_workspace_size(desc), dev)
    _check("hstu_layer_bwd", load_library().hstu_layer_bwd(
        ctypes.byref(desc), _ptr(x), _ptr(w1), _ptr(b1), _ptr(w2), _ptr(ln_gamma), _ptr(ln_beta),
        _ptr(seq_offsets), _ptr(timestamps), _ptr(num_targets), _ptr(rab_pos), _ptr(rab_time),
        _ptr(saved_uvqk), _ptr(saved_o), _ptr(dy), _ptr(out["dx"]), _ptr(out["dw1"]), _ptr(out["db1"]),
        _ptr(out["dw2"]), _ptr(out["db2"]), _ptr(out["d_ln_gamma"]), _ptr(out["d_ln_beta"]),
        _ptr(out["d_rab_pos"]), _ptr(out["d_rab_time"]), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
        _stream(stream)))
    return out


def hstu_e4m3_weight_bytes(K: int, N: int) -> int:
    return int(load_library().hstu_e4m3_weight_bytes(int(K), int(N)))


def quantize_weight_e4m3(w, stream=None):
    """E4M3 weight pack of a bf16 weight w [K, N]: uint8 tensor holding the
    codes [N, K] and, from byte align256(N K), the float32 scales [N]."""
    _dev(w, "w", torch.bfloat16)
    K, N = w.shape
    pack = torch.empty(hstu_e4m3_weight_bytes(K, N), dtype=torch.uint8, device=w.device)
    _check("hstu_quantize_weight_e4m3", load_library().hstu_quantize_weight_e4m3(
        _ptr(w), ctypes.c_int32(K), ctypes.c_int32(N), _ptr(pack), _stream(stream)))
    return pack


def e4m3_pack_parts(pack, K: int, N: int):
    """(codes [N, K] uint8, scales [N] float32) views of a weight pack."""
    off = (N * K + 255) // 256 * 256
    return pack[:N * K].view(N, K), pack[off:off + 4 * N].view(torch.float32)


def quantize_rows_e4m3(x, stream=None):
    """Per-row E4M3 codes [R, K] (uint8) and scales [R] (float32) of a bf16 x [R, K]."""
    _dev(x, "x", torch.bfloat16)
    R, K = x.shape
    codes = torch.empty((R, K), dtype=torch.uint8, device=x.device)
    scales = torch.empty(R, dtype=torch.float32, device=x.device)
    _check("hstu_quantize_rows_e4m3", load_library().hstu_quantize_rows_e4m3(
        _ptr(x), ctypes.c_int64(R), ctypes.c_int32(K), _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def gemm_e4m3(codes, scales, wpack, N: int, bias=None, apply_silu: bool = False, y=None, workspace=None,
              stream=None):
    """bf16 y [M, N] = dequant(codes, scales) dequant(W)^T + bias (optionally SiLU)."""
    _dev(codes, "codes", torch.uint8)
    _dev(scales, "scales", torch.float32)
    _dev(wpack, "wpack", torch.uint8)
    _dev(bias, "bias", torch.bfloat16)
    M, K = codes.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=codes.device)
    if workspace is None:
        workspace = alloc_workspace(256, codes.device)
    _check("hstu_gemm_e4m3", load_library().hstu_gemm_e4m3(
        _ptr(codes), _ptr(scales), ctypes.c_int64(M), ctypes.c_int32(K), _ptr(wpack), ctypes.c_int32(N),
        _ptr(bias), ctypes.c_int32(int(apply_silu)), _ptr(y), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
        _stream(stream)))
    return y


def hstu_jagged_truncate(seq_offsets, num_targets, keep: int, rows, *, out=None, out_offsets=None,
                         stream=None):
    """Attention truncation gather: each sequence's last min(hist, keep) history
    rows and all its candidates.  `rows` is any contiguous per-token tensor
    [T, ...] on the device.  Returns (out_offsets [B+1] int64, out) with `out`
    shaped like `rows` (T rows of room; the kept batch is out[:out_offsets[-1]])."""
    _dev(seq_offsets, "seq_offsets", torch.int64)
    _dev(num_targets, "num_targets", torch.int32)
    _dev(rows, "rows")
    B, T = seq_offsets.numel() - 1, rows.shape[0]
    row_bytes = rows.element_size() * math.prod(rows.shape[1:])
    if out is None:
        out = torch.empty_like(rows)
    if out_offsets is None:
        out_offsets = torch.empty(B + 1, dtype=torch.int64, device=rows.device)
    _dev(out, "out", rows.dtype)
    _dev(out_offsets, "out_offsets", torch.int64)
    _check("hstu_jagged_truncate", load_library().hstu_jagged_truncate(
        ctypes.c_int32(B), ctypes.c_int64(T), ctypes.c_int32(keep), _ptr(seq_offsets), _ptr(num_targets),
        _ptr(rows), ctypes.c_int64(row_bytes), _ptr(out), _ptr(out_offsets), _stream(stream)))
    return out_offsets, out


class HstuCache:
    """The tensors of an 8-bit key/value cache (layouts in include/hstu.h): E4M3 codes
    k_codes [pages, H, 64, d] and v_codes [pages, H, d, 64] (uint8), their scales
    [pages, H] (float32), and per token timestamps (int64), positions (int32) and
    optionally weights (float32), all [pages, 64] on one CUDA device."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, timestamps, positions, weights=None):
        pages, heads, page, d = k_codes.shape
        if page != HSTU_CACHE_PAGE:
            raise ValueError(f"k_codes has pages of {page} tokens, not {HSTU_CACHE_PAGE}")
        for name, t, dtype, shape in (("k_codes", k_codes, torch.uint8, (pages, heads, page, d)),
                                      ("v_codes", v_codes, torch.uint8, (pages, heads, d, page)),
                                      ("k_scale", k_scale, torch.float32, (pages, heads)),
                                      ("v_scale", v_scale, torch.float32, (pages, heads)),
                                      ("timestamps", timestamps, torch.int64, (pages, page)),
                                      ("positions", positions, torch.int32, (pages, page)),
                                      ("weights", weights, torch.float32, (pages, page))):
            if t is None:
                continue
            _dev(t, name, dtype)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
            _same_device(t, name, k_codes.device)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.timestamps, self.positions, self.weights = timestamps, positions, weights
        self.num_pages, self.num_heads, self.head_dim = int(pages), int(heads), int(d)
        self.device, self.device_index = k_codes.device, k_codes.get_device()
        self._structs = {}

    def __setattr__(self, name, value):
        if hasattr(self, "_structs"):  # the C structs hold the tensors' addresses
            raise AttributeError("a cache keeps its tensors; make another HstuCache")
        object.__setattr__(self, name, value)

    @classmethod
    def empty(cls, num_pages: int, num_heads: int, head_dim: int, device, weights: bool = True) -> "HstuCache":
        """A cache of num_pages pages, all zero."""
        def z(shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=device)

        pages, tokens = (num_pages, num_heads), (num_pages, HSTU_CACHE_PAGE)
        return cls(z(pages + (HSTU_CACHE_PAGE, head_dim), torch.uint8), z(pages + (head_dim, HSTU_CACHE_PAGE), torch.uint8),
                   z(pages, torch.float32), z(pages, torch.float32), z(tokens, torch.int64), z(tokens, torch.int32),
                   z(tokens, torch.float32) if weights else None)

    def struct(self, max_pages: int):
        """The C struct of these tensors with block tables of max_pages columns, by reference."""
        if max_pages not in self._structs:
            self._structs[max_pages] = ctypes.byref(hstu_cache(
                self.num_pages, self.num_heads, self.head_dim, int(max_pages), self.k_codes.data_ptr(),
                self.v_codes.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                self.timestamps.data_ptr(), self.positions.data_ptr(),
                0 if self.weights is None else self.weights.data_ptr()))
        return self._structs[max_pages]


def _same_device(t, name, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")


def _on(cache, t, name, dtype) -> int:
    """The address of a dense tensor of this type on the cache's device; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != cache.device_index or not t.is_contiguous():
        _dev(t, name, dtype)
        _same_device(t, name, cache.device)
    return t.data_ptr()


def _cache_table(cache, t, name, shape=None) -> int:
    p = _on(cache, t, name, torch.int32)
    if t is not None and (t.dim() != 2 if shape is None else t.shape != shape):
        raise ValueError(f"{name} must be [num_seqs, max_pages]")
    return p


def _cache_ints(cache, B, t, name) -> int:
    p = _on(cache, t, name, torch.int32)
    if t is not None and t.numel() != B:
        raise ValueError(f"{name} has {t.numel()} entries for {B} sequences")
    return p


def _cache_rows(cache, name, t):
    """Checks a [T, H, d] tensor whose rows may lie further apart than H * d; the row stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    H, d = cache.num_heads, cache.head_dim
    if t.dim() != 3 or t.shape[1] != H or t.shape[2] != d:
        raise ValueError(f"{name} must be [T, {H}, {d}], got {list(t.shape)}")
    st = t.stride()
    if t.numel() and (st[2] != 1 or (H > 1 and st[1] != d)):
        raise ValueError(f"{name} must have dense rows")
    if t.get_device() != cache.device_index:
        _same_device(t, name, cache.device)
    return st[0] if t.shape[0] > 1 else H * d


def _cache_tokens(cache, B, T, seq_offsets, timestamps):
    off = _on(cache, seq_offsets, "seq_offsets", torch.int64)
    ts = _on(cache, timestamps, "timestamps", torch.int64)
    if seq_offsets.numel() != B + 1 or timestamps.numel() != T:
        raise ValueError(f"seq_offsets needs {B + 1} entries and timestamps {T}")
    return off, ts


def _cache_empty(cache, stream, shape, dtype):
    """A new tensor on the stream of the call: the allocator gives its memory out again by that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=cache.device)
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                           torch.cuda.ExternalStream(_cache_stream(cache, stream), device=cache.device)):
        return torch.empty(shape, dtype=dtype, device=cache.device)


def _cache_workspace(cache, stream, workspace, need):
    if workspace is None:
        return _cache_empty(cache, stream, max(need, 256), torch.uint8)
    _same_device(workspace, "workspace", cache.device)
    return workspace


def _cache_call(cache, name, stream, *args):
    """Calls into the library on the cache's device and, by default, that device's current stream."""
    fn = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == cache.device_index:
        status = fn(*args, _cache_stream(cache, stream))
    else:
        with torch.cuda.device(cache.device):
            status = fn(*args, _cache_stream(cache, stream))
    _check(name, status)


def _cache_stream(cache, stream):
    if stream is None:  # the raw handle: a Stream object costs 2 us
        return torch._C._cuda_getCurrentRawStream(cache.device_index)
    if not hasattr(stream, "cuda_stream"):
        return int(stream)
    if stream.device != cache.device:
        raise ValueError(f"the stream is on {stream.device}, the cache on {cache.device}")
    return stream.cuda_stream


def hstu_cache_append_workspace_size() -> int:
    n = ctypes.c_size_t(0)
    _check("hstu_cache_append_workspace_size", load_library().hstu_cache_append_workspace_size(ctypes.byref(n)))
    return n.value


def hstu_cache_append(k, v, cache: HstuCache, block_table, cache_lens, seq_pos, seq_offsets, timestamps, num_targets, *,
                      max_seq_len: int, new_lens=None, new_pos=None, workspace=None, stream=None):
    """Append each sequence's history tokens to the cache: k, v [T, H, d] (rows may lie
    further apart, as in a projection's output).  Returns (new_lens, new_pos) [B] int32;
    seq_pos None means cache_lens (nothing was evicted before)."""
    table = _cache_table(cache, block_table, "block_table")
    B, cols = block_table.shape
    lens = _cache_ints(cache, B, cache_lens, "cache_lens")
    pos = _cache_ints(cache, B, seq_pos, "seq_pos")
    nt = _cache_ints(cache, B, num_targets, "num_targets")
    sk, sv = _cache_rows(cache, "k", k), _cache_rows(cache, "v", v)
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have one type and shape")
    T = k.shape[0]
    off, ts = _cache_tokens(cache, B, T, seq_offsets, timestamps)
    if new_lens is None:
        new_lens = _cache_empty(cache, stream, B, torch.int32)
    if new_pos is None:
        new_pos = _cache_empty(cache, stream, B, torch.int32)
    workspace = _cache_workspace(cache, stream, workspace, 256)
    _cache_call(cache, "hstu_cache_append", stream, cache.struct(cols), _dtype_code(k), B, int(max_seq_len), T, k.data_ptr(), sk,
                v.data_ptr(), sv, off, ts, nt, table, lens, pos, _cache_ints(cache, B, new_lens, "new_lens"),
                _cache_ints(cache, B, new_pos, "new_pos"), workspace.data_ptr(), workspace.numel())
    return new_lens, new_pos


def _cache_attn_desc(q, block_table, rab_pos, rab_time, max_seq_len, inv_n, pos_lo, pos_hi, cand_own_index):
    T, H, d = q.shape
    nb, per_head = _tables(rab_pos, rab_time, H, pos_lo, pos_hi)
    return hstu_attn_desc(block_table.shape[0], int(max_seq_len), T, H, d, d, _dtype_code(q), inv_n, int(pos_lo),
                          int(pos_hi), nb, 0, 0, 0, 0, bool(cand_own_index), per_head)


def hstu_cache_attn_workspace_size(q, cache: HstuCache, block_table, rab_pos, rab_time, *, max_seq_len: int,
                                   max_cache_len: int, inv_n: float, pos_lo: int, pos_hi: int,
                                   cand_own_index: bool = False, weights: bool = False) -> int:
    desc = _cache_attn_desc(q, block_table, rab_pos, rab_time, max_seq_len, inv_n, pos_lo, pos_hi, cand_own_index)
    n = ctypes.c_size_t(0)
    _check("hstu_cache_attn_workspace_size", load_library().hstu_cache_attn_workspace_size(
        ctypes.byref(desc), cache.struct(block_table.shape[1]), int(max_cache_len), int(weights), ctypes.byref(n)))
    return n.value


def hstu_cache_attn_fwd(q, cache: HstuCache, block_table, cache_lens, seq_pos, seq_offsets, timestamps, num_targets,
                        rab_pos, rab_time, *, max_seq_len: int, max_cache_len: int, inv_n: float, pos_lo: int,
                        pos_hi: int, addend=None, weights_out=None, out=None, workspace=None, stream=None,
                        cand_own_index: bool = False):
    """Attention of q [T, H, d] over the sequences' whole caches, plus `addend` [T, H, d]
    (hstu_attn_fwd over the new tokens themselves; may be `out`).  weights_out
    [pages, 64] float32 receives the cached tokens' accumulated attention weight; it
    may be cache.weights."""
    table = _cache_table(cache, block_table, "block_table")
    B, cols = block_table.shape
    lens = _cache_ints(cache, B, cache_lens, "cache_lens")
    pos = _cache_ints(cache, B, seq_pos, "seq_pos")
    nt = _cache_ints(cache, B, num_targets, "num_targets")
    sq = _cache_rows(cache, "q", q)
    off, ts = _cache_tokens(cache, B, q.shape[0], seq_offsets, timestamps)
    rp = _on(cache, rab_pos, "rab_pos", torch.float32)
    rt = _on(cache, rab_time, "rab_time", torch.float32)
    if out is None:
        out = _cache_empty(cache, stream, q.shape, q.dtype)
    for name, t in (("addend", addend), ("out", out)):
        if t is not None and t.shape != q.shape:
            raise ValueError(f"{name} must have q's shape")
    if weights_out is not None and tuple(weights_out.shape) != (cache.num_pages, HSTU_CACHE_PAGE):
        raise ValueError("weights_out must be [pages, 64]")
    desc = ctypes.byref(_cache_attn_desc(q, block_table, rab_pos, rab_time, max_seq_len, inv_n, pos_lo, pos_hi,
                                         cand_own_index))
    pool = cache.struct(cols)
    need = 0
    if workspace is None:
        n = ctypes.c_size_t(0)
        with torch.cuda.device(cache.device):
            _check("hstu_cache_attn_workspace_size", load_library().hstu_cache_attn_workspace_size(
                desc, pool, int(max_cache_len), int(weights_out is not None), ctypes.byref(n)))
        need = n.value
    workspace = _cache_workspace(cache, stream, workspace, need)
    _cache_call(cache, "hstu_cache_attn_fwd", stream, desc, pool, int(max_cache_len), q.data_ptr(), sq, off, ts, nt, rp, rt,
                table, lens, pos, _on(cache, addend, "addend", q.dtype),
                _on(cache, weights_out, "weights_out", torch.float32), _on(cache, out, "out", q.dtype),
                workspace.data_ptr(), workspace.numel())
    return out


def hstu_cache_evict_workspace_size(cache: HstuCache, block_table, *, keep: int, max_cache_len: int, first: int = 0,
                                    recent: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check("hstu_cache_evict_workspace_size", load_library().hstu_cache_evict_workspace_size(
        cache.struct(block_table.shape[1]), block_table.shape[0], int(max_cache_len), int(keep), ctypes.byref(n)))
    return n.value


def hstu_cache_evict(cache: HstuCache, block_table, cache_lens, new_pages, *, keep: int, max_cache_len: int,
                     first: int = 0, recent: int = 0, new_table=None, new_lens=None, kept=None, workspace=None,
                     stream=None):
    """Cut every sequence of more than `keep` tokens to its first `first`, its last
    `recent` and, of the rest, the tokens of largest weight; they move into the pages
    of new_pages [B, max_pages].  Returns (new_table, new_lens, kept [B, keep])."""
    table = _cache_table(cache, block_table, "block_table")
    B, cols = block_table.shape
    keep = int(keep)
    if cache.weights is None:
        raise ValueError("eviction needs the cache's weights")
    if new_table is None:
        new_table = _cache_empty(cache, stream, (B, cols), torch.int32)
    if new_lens is None:
        new_lens = _cache_empty(cache, stream, B, torch.int32)
    if kept is None:
        kept = _cache_empty(cache, stream, (B, keep), torch.int32)
    if tuple(kept.shape) != (B, keep):
        raise ValueError(f"kept must be [{B}, {keep}]")
    need = 0 if workspace is not None else hstu_cache_evict_workspace_size(cache, block_table, keep=keep,
                                                                           max_cache_len=max_cache_len)
    workspace = _cache_workspace(cache, stream, workspace, need)
    _cache_call(cache, "hstu_cache_evict", stream, cache.struct(cols), B, int(max_cache_len), keep, int(first), int(recent), table,
                _cache_ints(cache, B, cache_lens, "cache_lens"),
                _cache_table(cache, new_pages, "new_pages", block_table.shape),
                _cache_table(cache, new_table, "new_table", block_table.shape),
                _cache_ints(cache, B, new_lens, "new_lens"), _on(cache, kept, "kept", torch.int32),
                workspace.data_ptr(), workspace.numel())
    return new_table, new_lens, kept


def hstu_check_device_flag(workspace: torch.Tensor, stream=None):
    """(status, bits) of the device input check of the last call on `workspace`."""
    bits = ctypes.c_int32(0)
    st = load_library().hstu_check_device_flag(_ptr(workspace), ctypes.byref(bits), _stream(stream))
    return st, bits.value


def hstu_debug_bias_indices(desc: hstu_attn_desc, seq_offsets, timestamps, num_targets, rows,
                            stream=None):
    n = rows.shape[0]
    pos = torch.empty(n, dtype=torch.int32, device=rows.device)
    bkt = torch.empty(n, dtype=torch.int32, device=rows.device)
    _check("hstu_debug_bias_indices", load_library().hstu_debug_bias_indices(
        ctypes.byref(desc), _ptr(seq_offsets), _ptr(timestamps), _ptr(num_targets), _ptr(rows),
        ctypes.c_int64(n), _ptr(pos), _ptr(bkt), _stream(stream)))
    return pos, bkt


def hstu_debug_schedule(desc: hstu_attn_desc, seq_offsets, num_targets, is_bwd: bool,
                        tile_rows: int, stream=None):
    T, B = desc.total_tokens, desc.num_seqs
    cap = (T + tile_rows - 1) // tile_rows + B
    dev = seq_offsets.device
    items = torch.full((max(cap, 1), 2), -1, dtype=torch.int32, device=dev)
    count = torch.zeros(1, dtype=torch.int32, device=dev)
    hdr = torch.zeros(64, dtype=torch.int32, device=dev)
    _check("hstu_debug_schedule", load_library().hstu_debug_schedule(
        ctypes.byref(desc), _ptr(seq_offsets), _ptr(num_targets), int(is_bwd), int(tile_rows),
        _ptr(items), ctypes.c_int32(cap), _ptr(count), _ptr(hdr), _stream(stream)))
    return items, count, hdr
