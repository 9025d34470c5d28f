"""GB300-native tensor-parallel sharded projections: a thin binding over libtp.so.

Every function here has the name of the C entry point it calls (see
``include/tp.h``) and does argument marshalling only: it checks dtypes,
allocates outputs with PyTorch when the caller passes none, and hands raw
pointers and the current CUDA stream to the library.  All computation runs in
the library's CUDA kernels; there is no other path.  If ``libtp.so`` has not
been built, importing this package raises ImportError.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtp.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python tensor_sharded_linear_tp_gb300/build.py` "
        "(the CUDA library is the only implementation)")

lib = ctypes.CDLL(LIB_PATH)

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_status = ctypes.c_int

# Status codes and enums, mirrored from include/tp.h.
TP_OK = 0
STATUS_NAMES = ["TP_OK", "TP_ERR_INVALID_ARG", "TP_ERR_HEADS_NOT_DIVISIBLE", "TP_ERR_SPLIT_NOT_DIVISIBLE",
                "TP_ERR_SPLIT_SUM", "TP_ERR_NOT_WHOLE_HEADS", "TP_ERR_ALIGNMENT", "TP_ERR_NOT_PINNED",
                "TP_ERR_WORKSPACE", "TP_ERR_CUDA", "TP_ERR_TIMEOUT", "TP_ERR_UNSUPPORTED", "TP_ERR_IO",
                "TP_ERR_FORMAT", "TP_ERR_NOT_FOUND"]
STYLES = {"colwise": 0, "rowwise": 1}
ACTS = {"none": 0, "gelu_tanh": 1, "swiglu": 2}
ACCUM_CHUNKED = 0x100   # TP_ACCUM_CHUNKED (include/tp.h): OR'd into the colwise act argument
REDUCE_MODES = {"none": 0, "workspace": 1, "accum": 2}
COMBINE_MODES = {"gather": 0, "reduce": 1}
NORMS = {"none": 0, "rms": 1, "layer": 2}
FP8_GROUP = 128         # features (or weight rows) that share a scale
NORM_MAX_D = 32768      # TP_NORM_MAX_D
ROPE_STYLES = {"half": 0, "pairs": 1}
MAX_DEGREE = 16
MAX_SPLITS = 16

_SIGS = {
    "tp_validate": (_status, [_i64, _i64, ctypes.c_int, ctypes.c_int, _i64, _i64, ctypes.POINTER(_i64), ctypes.c_int]),
    "tp_shard_shape": (_status, [_i64, _i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(_i64), ctypes.c_int,
                                 ctypes.POINTER(_i64), ctypes.POINTER(_i64)]),
    "tp_plan_shard": (_status, [_vp, _i64, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(_i64),
                                ctypes.c_int, _i64, _i64, _vp, _vp]),
    "tp_plan_shard_ranks": (_status, [_vp, _i64, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.POINTER(_i64), ctypes.c_int, _i64, _i64, ctypes.POINTER(_vp), _vp]),
    "tp_linear_colwise": (_status, [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int, ctypes.c_int, _i64,
                                    _i64, _i64, ctypes.POINTER(_vp), _i64, _vp]),
    "tp_linear_rowwise": (_status, [ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp, ctypes.c_int, _i64, _i64, _i64,
                                    ctypes.c_int, _vp, ctypes.c_size_t, _vp, _vp]),
    "tp_linear_rowwise_split_input": (_status, [_vp, _i64, ctypes.POINTER(_vp), _vp, ctypes.c_int, _i64, _i64, _i64,
                                                ctypes.c_int, _vp, ctypes.c_size_t, _vp, _vp]),
    "tp_linear_rowwise_noalloc": (_status, [ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp, ctypes.c_int, _i64, _i64,
                                            _i64, _vp, _vp]),
    "tp_rowwise_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, _i64, _i64, ctypes.c_int]),
    "tp_attention_heads": (_status, [_vp, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp, ctypes.c_size_t, _vp, _i64,
                                     _vp]),
    "tp_attention_workspace_bytes": (ctypes.c_size_t, [_i64, ctypes.c_int, ctypes.c_int]),
    "tp_attention_heads_ranks": (_status, [ctypes.c_int, ctypes.POINTER(_vp), _i64, _i64, ctypes.c_int, ctypes.c_int,
                                           _vp, ctypes.c_size_t, ctypes.POINTER(_vp), _i64, _vp]),
    "tp_attention_ranks_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int]),
    "tp_combine": (_status, [ctypes.c_int, ctypes.POINTER(_vp), ctypes.c_int, _i64, _i64, _vp, _vp]),
    "tp_quantize_fp8": (_status, [_vp, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _i64, _vp]),
    # (their arrays of pointers are passed as bytes, see _pointers)
    "tp_linear_colwise_fp8": (_status, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, ctypes.c_int, ctypes.c_int, _i64, _i64,
                                        _i64, _vp, _i64, _vp, _i64, _vp]),
    "tp_linear_rowwise_fp8": (_status, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, ctypes.c_int, _i64, _i64, _i64, _vp,
                                        _i64, _vp]),
    # (their structures and arrays of pointers are passed as bytes, see PagedCache)
    "tp_kv_append_fp8": (_status, [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _vp, _vp, _i64, _vp]),
    "tp_attention_paged_fp8": (_status, [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, ctypes.c_float, ctypes.c_int,
                                         ctypes.c_int, _vp, ctypes.c_size_t, _vp, _i64, _vp]),
    "tp_attention_paged_workspace_bytes": (ctypes.c_size_t, [_vp, _vp, _i64, ctypes.c_int]),
    "tp_last_error": (ctypes.c_char_p, []),
    "tp_status_name": (ctypes.c_char_p, [ctypes.c_int]),
    "tp_device_status": (_status, [_vp]),
    "tp_abi_version": (ctypes.c_int, []),
    "tp_set_tile_wait_limit_ns": (None, [ctypes.c_uint64]),
    "tp_tile_wait_limit_ns": (ctypes.c_uint64, []),
    # include/tp_safetensors.h
    "tp_st_dtype_size": (ctypes.c_size_t, [ctypes.c_int]),
    "tp_st_open": (_status, [ctypes.c_char_p, ctypes.c_size_t, ctypes.POINTER(_vp)]),
    "tp_st_close": (_status, [_vp]),
    "tp_st_set_read_mode": (_status, [_vp, ctypes.c_int]),
    "tp_st_read_mode_on_device": (_status, [_vp, ctypes.POINTER(ctypes.c_int)]),
    "tp_st_count": (_i64, [_vp]),
    "tp_st_info": (_status, [_vp, _i64, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_int),
                             ctypes.POINTER(ctypes.c_int), ctypes.POINTER(_i64), ctypes.POINTER(ctypes.c_uint64),
                             ctypes.POINTER(ctypes.c_uint64)]),
    "tp_st_find": (_i64, [_vp, ctypes.c_char_p]),
    "tp_st_plan_shard_ranks": (_status, [_vp, ctypes.c_char_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.POINTER(_i64), ctypes.c_int, _i64, _i64, ctypes.POINTER(_vp), _vp]),
}
class ShardRequest(ctypes.Structure):
    """Mirror of tp_shard_request (include/tp.h)."""
    _fields_ = [("weight", _vp), ("rows", _i64), ("cols", _i64), ("style", ctypes.c_int), ("tp_degree", ctypes.c_int),
                ("rank_begin", ctypes.c_int), ("rank_count", ctypes.c_int), ("fused_splits", ctypes.POINTER(_i64)),
                ("n_splits", ctypes.c_int), ("num_heads", _i64), ("head_dim", _i64),
                ("dev_outs", ctypes.POINTER(_vp))]


class ResidualNormArgs(ctypes.Structure):
    """Mirror of tp_residual_norm_args (include/tp.h)."""
    _fields_ = [("T", _i64), ("D", _i64), ("x", _vp), ("ldx", _i64), ("y", _vp), ("ldy", _i64),
                ("post_norm", ctypes.c_int), ("post_weight", _vp), ("post_bias", _vp), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("gate", _vp), ("scale", _vp), ("shift", _vp), ("ld_mod", _i64),
                ("mod_rows", _i64), ("rows_per_mod", _i64), ("h", _vp), ("ldh", _i64), ("norm", ctypes.c_int),
                ("weight", _vp), ("bias", _vp), ("u", _vp), ("ldu", _i64), ("u_scales", _vp), ("ld_u_scales", _i64)]


_SIGS["tp_plan_shard_many"] = (_status, [ctypes.POINTER(ShardRequest), ctypes.c_int, _vp])
_SIGS["tp_residual_norm"] = (_status, [_vp, _vp])
# The same structure as bytes, in native alignment (q: int64, P: pointer, i: enum).
_residual_norm_args = struct.Struct("@qq PqPq iPP ff PPP qqq Pq iPP PqPq").pack
_paged_cache = struct.Struct("@iiii q PPPP qq").pack      # tp_paged_cache
_paged_batch = struct.Struct("@ii PPP qq").pack           # tp_paged_batch
_rope = struct.Struct("@iiPqqP").pack                     # tp_rope

for _name, (_res, _args) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


class TPError(RuntimeError):
    """A libtp call returned a status other than TP_OK."""

    def __init__(self, status: int, message: str):
        self.status = status
        self.name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else f"status {status}"
        super().__init__(message or self.name)


def _check(status: int) -> None:
    if status != TP_OK:
        raise TPError(status, lib.tp_last_error().decode())


def _splits(fused_splits):
    if not fused_splits:
        return None, 0
    arr = (_i64 * len(fused_splits))(*[int(s) for s in fused_splits])
    return arr, len(fused_splits)


def _ptrs(tensors):
    return (_vp * len(tensors))(*[_ptr(t) for t in tensors])


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        if not torch.cuda.is_available():
            return None
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need_bf16(name, t):
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_bf16_rows(name, t):
    """bf16 2-D with contiguous rows (any row stride): the library takes the stride."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must be 2-D with contiguous rows")


# ---------------------------------------------------------------------------
# Plan
# ---------------------------------------------------------------------------

def tp_validate(rows: int, cols: int, style: str, tp_degree: int, num_heads: int = 0, head_dim: int = 0,
                fused_splits: Sequence[int] | None = None) -> None:
    """Raise TPError unless the plan is valid (tp_degree divides the heads, blocks divide, whole heads)."""
    arr, n = _splits(fused_splits)
    _check(lib.tp_validate(rows, cols, STYLES[style], tp_degree, num_heads, head_dim, arr, n))


def tp_shard_shape(rows: int, cols: int, style: str, tp_degree: int,
                   fused_splits: Sequence[int] | None = None) -> tuple[int, int]:
    arr, n = _splits(fused_splits)
    r, c = _i64(), _i64()
    _check(lib.tp_shard_shape(rows, cols, STYLES[style], tp_degree, arr, n, ctypes.byref(r), ctypes.byref(c)))
    return r.value, c.value


# ---------------------------------------------------------------------------
# Shard extraction
# ---------------------------------------------------------------------------

def tp_plan_shard(weight: torch.Tensor, style: str, tp_degree: int, rank: int,
                  fused_splits: Sequence[int] | None = None, num_heads: int = 0, head_dim: int = 0,
                  out: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """Rank ``rank``'s dense shard of a bf16 weight, on the GPU.

    ``weight`` is a bf16 [rows, cols] tensor in page-locked host memory
    (shard-on-read: only the slice crosses to the device) or on the GPU.
    """
    _need_bf16("weight", weight)
    rows, cols = weight.shape
    arr, n = _splits(fused_splits)
    if out is None:
        tp_validate(rows, cols, style, tp_degree, num_heads, head_dim, fused_splits)  # before allocating
        shape = tp_shard_shape(rows, cols, style, tp_degree, fused_splits)
        dev = device if device is not None else (weight.device if weight.is_cuda else torch.device("cuda"))
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _check(lib.tp_plan_shard(_ptr(weight), rows, cols, STYLES[style], tp_degree, rank, arr, n, num_heads, head_dim,
                             _ptr(out), _stream(stream)))
    return out


def tp_plan_shard_ranks(weight: torch.Tensor, style: str, tp_degree: int, rank_begin: int = 0,
                        rank_count: int | None = None, fused_splits: Sequence[int] | None = None, num_heads: int = 0,
                        head_dim: int = 0, outs: Sequence[torch.Tensor] | None = None, device=None,
                        stream=None) -> list[torch.Tensor]:
    """Shards of ranks [rank_begin, rank_begin + rank_count) in one launch (default: every rank)."""
    _need_bf16("weight", weight)
    rows, cols = weight.shape
    if rank_count is None:
        rank_count = tp_degree - rank_begin
    arr, n = _splits(fused_splits)
    if outs is None:
        tp_validate(rows, cols, style, tp_degree, num_heads, head_dim, fused_splits)  # before allocating
        shape = tp_shard_shape(rows, cols, style, tp_degree, fused_splits)
        dev = device if device is not None else (weight.device if weight.is_cuda else torch.device("cuda"))
        outs = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(rank_count)]
    _check(lib.tp_plan_shard_ranks(_ptr(weight), rows, cols, STYLES[style], tp_degree, rank_begin, rank_count, arr, n,
                                   num_heads, head_dim, _ptrs(outs) if outs else None, _stream(stream)))
    return list(outs)


# ---------------------------------------------------------------------------
# Projections
# ---------------------------------------------------------------------------

def tp_plan_shard_many(requests: Sequence[dict], device=None, stream=None) -> list[list[torch.Tensor]]:
    """Several tp_plan_shard_ranks extractions in as few launches as possible.

    Each request is a dict with keys weight, style, tp_degree and optionally rank_begin,
    rank_count, fused_splits, num_heads, head_dim, outs (as for tp_plan_shard_ranks).
    Every request is checked before anything is copied.  Returns each request's outputs.
    """
    keep = []
    arr = (ShardRequest * max(1, len(requests)))()
    all_outs = []
    for i, rq in enumerate(requests):
        w = rq["weight"]
        _need_bf16("weight", w)
        rows, cols = w.shape
        style, p = rq["style"], rq["tp_degree"]
        rb = rq.get("rank_begin", 0)
        rc = rq.get("rank_count")
        rc = p - rb if rc is None else rc
        splits = rq.get("fused_splits")
        heads, hd = rq.get("num_heads", 0), rq.get("head_dim", 0)
        outs = rq.get("outs")
        if outs is None:
            tp_validate(rows, cols, style, p, heads, hd, splits)  # before allocating
            shape = tp_shard_shape(rows, cols, style, p, splits)
            dev = device if device is not None else (w.device if w.is_cuda else torch.device("cuda"))
            outs = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(rc)]
        sp, n = _splits(splits)
        ptrs = _ptrs(outs) if outs else None
        keep += [sp, ptrs]
        arr[i] = ShardRequest(_ptr(w), rows, cols, STYLES[style], p, rb, rc, sp, n, heads, hd, ptrs)
        all_outs.append(list(outs))
    _check(lib.tp_plan_shard_many(arr, len(requests), _stream(stream)))
    return all_outs


def tp_linear_colwise(x: torch.Tensor, w_shards: Sequence[torch.Tensor], act: str = "none",
                      bias_shards: Sequence[torch.Tensor | None] | None = None,
                      y_shards: Sequence[torch.Tensor] | None = None, ldy: int = 0, stream=None,
                      chunked: bool = False):
    """Y_r = act(X W_r^T + b_r) for every rank r, one launch.  Returns the list of Y_r.

    chunked=True (act "none" only): the K sum is formed in chunks of 1024 on the tensor core and
    the chunks are added with round-to-nearest (TP_ACCUM_CHUNKED), for outputs that feed
    attention."""
    _need_bf16("x", x)
    p = len(w_shards)
    T, K = x.shape
    N_r = w_shards[0].shape[0]
    for w in w_shards:
        _need_bf16("w_shards[i]", w)
    n_out = N_r // 2 if act == "swiglu" else N_r
    if y_shards is None:
        y_shards = [torch.empty((T, n_out), dtype=torch.bfloat16, device=x.device) for _ in range(p)]
    bias_arr = _ptrs(bias_shards) if bias_shards is not None else None
    code = ACTS[act] | (ACCUM_CHUNKED if chunked else 0)
    _check(lib.tp_linear_colwise(_ptr(x), _ptrs(w_shards), bias_arr, code, p, T, K, N_r, _ptrs(y_shards), ldy,
                                 _stream(stream)))
    return y_shards


def tp_rowwise_workspace_bytes(tp_degree: int, T: int, N: int, mode: str = "workspace") -> int:
    return int(lib.tp_rowwise_workspace_bytes(tp_degree, T, N, REDUCE_MODES[mode]))


def tp_linear_rowwise(x_shards: Sequence[torch.Tensor], w_shards: Sequence[torch.Tensor],
                      bias: torch.Tensor | None = None, mode: str = "accum", workspace: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Z = sum_r X_r W_r^T (+ bias once), one launch.

    mode "accum" / "workspace" return bf16 [T, N]; "none" returns the fp32
    partials [tp_degree, T, N] (join them with ``tp_combine("reduce", ...)``).
    """
    p = len(w_shards)
    T, K_r = x_shards[0].shape
    N = w_shards[0].shape[0]
    for t in list(x_shards) + list(w_shards):
        _need_bf16("shard", t)
    dev = x_shards[0].device
    if out is None:
        if mode == "none":
            out = torch.empty((p, T, N), dtype=torch.float32, device=dev)
        else:
            out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    need = tp_rowwise_workspace_bytes(p, T, N, mode)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.tp_linear_rowwise(_ptrs(x_shards), _ptrs(w_shards), _ptr(bias), p, T, K_r, N, REDUCE_MODES[mode],
                                 _ptr(workspace), ws_bytes, _ptr(out), _stream(stream)))
    return out


def tp_linear_rowwise_split_input(x: torch.Tensor, w_shards: Sequence[torch.Tensor], bias: torch.Tensor | None = None,
                                  mode: str = "accum", workspace: torch.Tensor | None = None,
                                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Z = sum_r X[:, r*K/p:(r+1)*K/p] W_r^T (+ bias once): each rank slices the replicated input itself."""
    _need_bf16_rows("x", x)
    p = len(w_shards)
    T, K = x.shape
    N = w_shards[0].shape[0]
    if out is None:
        shape = (p, T, N) if mode == "none" else (T, N)
        out = torch.empty(shape, dtype=torch.float32 if mode == "none" else torch.bfloat16, device=x.device)
    need = tp_rowwise_workspace_bytes(p, T, N, mode)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.tp_linear_rowwise_split_input(_ptr(x), x.stride(0), _ptrs(w_shards), _ptr(bias), p, T, K, N,
                                             REDUCE_MODES[mode], _ptr(workspace), ws_bytes, _ptr(out),
                                             _stream(stream)))
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def tp_linear_rowwise_noalloc(x_shards: Sequence[torch.Tensor], w_shards: Sequence[torch.Tensor],
                              bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """Rowwise projection with the summed partials, using the library's built-in scratch.

    For callers that may not allocate device memory: the fp32 partials live in
    a fixed 64 MiB array inside libtp.so instead of a caller workspace.  Only
    ``out`` (bf16 [T, N]) is allocated here, and only when none is passed.
    Calls that overlap on the GPU share that array and must be serialised.
    """
    p = len(w_shards)
    T, K_r = x_shards[0].shape
    N = w_shards[0].shape[0]
    for t in list(x_shards) + list(w_shards):
        _need_bf16("shard", t)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=x_shards[0].device)
    _check(lib.tp_linear_rowwise_noalloc(_ptrs(x_shards), _ptrs(w_shards), _ptr(bias), p, T, K_r, N, _ptr(out),
                                         _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# Attention over a rank's local heads
# ---------------------------------------------------------------------------

def tp_attention_workspace_bytes(T: int, n_heads: int, head_dim: int) -> int:
    return int(lib.tp_attention_workspace_bytes(T, n_heads, head_dim))


def tp_attention_heads(qkv: torch.Tensor, n_heads: int, head_dim: int, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """softmax(Q_h K_h^T / sqrt(d)) V_h for each local head of a rank's QKV output [T, 3*n_heads*d]."""
    _need_bf16_rows("qkv", qkv)
    T = qkv.shape[0]
    width = n_heads * head_dim
    if out is None:
        out = torch.empty((T, width), dtype=torch.bfloat16, device=qkv.device)
    need = tp_attention_workspace_bytes(T, n_heads, head_dim)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=qkv.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.tp_attention_heads(_ptr(qkv), qkv.stride(0), T, n_heads, head_dim, _ptr(workspace), ws_bytes,
                                  _ptr(out), out.stride(0), _stream(stream)))
    return out


def tp_attention_ranks_workspace_bytes(n_ranks: int, T: int, n_heads: int, head_dim: int) -> int:
    return int(lib.tp_attention_ranks_workspace_bytes(n_ranks, T, n_heads, head_dim))


def tp_attention_heads_ranks(qkv: Sequence[torch.Tensor], n_heads: int, head_dim: int,
                             outs: Sequence[torch.Tensor] | None = None, workspace: torch.Tensor | None = None,
                             stream=None) -> list[torch.Tensor]:
    """tp_attention_heads for every rank's QKV output in one call (one launch at head_dim 64 or 128)."""
    n = len(qkv)
    for t in qkv:
        _need_bf16_rows("qkv[r]", t)
    if len({t.stride(0) for t in qkv}) != 1:
        raise ValueError("every rank's qkv must have the same row stride")
    T = qkv[0].shape[0]
    width = n_heads * head_dim
    if outs is None:
        outs = [torch.empty((T, width), dtype=torch.bfloat16, device=qkv[0].device) for _ in range(n)]
    if len({t.stride(0) for t in outs}) != 1:
        raise ValueError("every rank's output must have the same row stride")
    need = tp_attention_ranks_workspace_bytes(n, T, n_heads, head_dim)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=qkv[0].device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.tp_attention_heads_ranks(n, _ptrs(qkv), qkv[0].stride(0), T, n_heads, head_dim, _ptr(workspace),
                                        ws_bytes, _ptrs(outs), outs[0].stride(0), _stream(stream)))
    return list(outs)


# ---------------------------------------------------------------------------
# Join
# ---------------------------------------------------------------------------

def tp_combine(mode: str, partials: Sequence[torch.Tensor], out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Gather bf16 [T, N_each] slices into [T, p*N_each], or reduce fp32 partials into bf16 [T, N_each]."""
    p = len(partials)
    T, N_each = partials[0].shape
    if out is None:
        cols = N_each * p if mode == "gather" else N_each
        out = torch.empty((T, cols), dtype=torch.bfloat16, device=partials[0].device)
    _check(lib.tp_combine(COMBINE_MODES[mode], _ptrs(partials), p, T, N_each, _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# 8-bit projections and the residual norm
#
# The block-scaled format (include/tp.h): float8_e4m3fn codes with one power-of-two scale per
# group of 128, a float8_e8m0fnu (or uint8) byte.  These calls check every tensor's type, shape,
# strides and device before the library is called, so a refused call touches no device memory.
# ---------------------------------------------------------------------------

_E4M3, _E8M0, _BF16, _U8 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16, torch.uint8
# A host array of n device pointers, as the bytes of one (made in a fifth of the time of a ctypes array).
_pointers = [struct.Struct(f"{n}P").pack for n in range(MAX_DEGREE + 1)]


def _groups(n: int) -> int:
    return -(-n // FP8_GROUP)


def _need(name, t, dtype, shape, dev):
    """A tensor of `dtype` (a scale: e8m0 or uint8) and `shape` on the current GPU, its last dimension contiguous.

    Returns the row stride (0 where the rows are dense)."""
    if t.dtype is dtype and t.is_contiguous() and t.shape == shape and t.get_device() == dev:
        return 0
    if t.dtype is not dtype and not (dtype is _E8M0 and t.dtype is _U8):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    if t.is_contiguous():
        return 0
    if len(shape) == 1:
        raise ValueError(f"{name} must be contiguous")
    rows, cols = shape
    step, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows > 1 and step < cols:
        raise ValueError(f"{name}: a row stride of {step} overlaps rows of {cols} elements")
    return step if rows > 1 else 0


def _need_ranks(name, ts, dtype, shape, dev, dense=False):
    """(pointer array, row stride) of one tensor for each rank, as _need; every rank has the same row stride."""
    at = []
    for t in ts:   # the usual case, in as few steps as it takes: a call with few tokens is as long as its checks
        if t.dtype is not dtype or not t.is_contiguous() or t.shape != shape or t.get_device() != dev:
            break
        at.append(t.data_ptr())
    else:
        return _pointers[len(at)](*at), 0
    steps = [_need(f"{name}[{i}]", t, dtype, shape, dev) for i, t in enumerate(ts)]
    if any(s not in (0, shape[-1]) for s in steps):
        if dense:
            raise ValueError(f"every rank's {name} must be contiguous")
        if any(s != steps[0] for s in steps):
            raise ValueError(f"every rank's {name} must have the same row stride")
    return _pointers[len(ts)](*[t.data_ptr() for t in ts]), steps[0]


def _alloc(stream, device, dtype, shape, count=1):
    """`count` outputs for a call on `stream`, from that stream's memory."""
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return _alloc(None, device, dtype, shape, count)
    # (One by one: 1.5 us each on the host, where views of one allocation take 2 to 7.)
    return [torch.empty(shape, dtype=dtype, device=device) for _ in range(count)]


def _launch_stream(stream, dev) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _device_of(name, t) -> int:
    """The current device, which a 2-D tensor `t` has to be on."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    return dev


def _ranks(w_shards, *lists) -> int:
    p = len(w_shards)
    if p < 1 or p > MAX_DEGREE:
        raise ValueError(f"w_shards must have one entry for each of 1 to {MAX_DEGREE} ranks, got {p}")
    for ts in lists:
        if ts is not None and len(ts) != p:
            raise ValueError(f"every list must have one entry for each of the {p} ranks, got {len(ts)}")
    return p


def tp_quantize_fp8(x: torch.Tensor, block_rows: int = 1, q: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of a bf16 [rows, cols]: groups of 1 x 128 (activations) or 128 x 128 (weights)."""
    dev = _device_of("x", x)
    if block_rows not in (1, FP8_GROUP):
        raise ValueError(f"block_rows must be 1 or {FP8_GROUP}, got {block_rows}")
    shape = x.shape
    rows, cols = shape
    ldx = 0 if x.dtype is _BF16 and x.is_contiguous() else _need("x", x, _BF16, shape, dev)
    s_shape = (-(-rows // block_rows), _groups(cols))
    if q is None:
        q, = _alloc(stream, x.device, _E4M3, shape)
    if scales is None:
        scales, = _alloc(stream, x.device, _E8M0, s_shape)
    ldq, lds = _need("q", q, _E4M3, shape, dev), _need("scales", scales, _E8M0, s_shape, dev)
    _check(lib.tp_quantize_fp8(x.data_ptr(), ldx, rows, cols, block_rows, q.data_ptr(), ldq, scales.data_ptr(), lds,
                               _launch_stream(stream, dev)))
    return q, scales


def tp_linear_colwise_fp8(x: torch.Tensor, x_scales: torch.Tensor, w_shards: Sequence[torch.Tensor],
                          w_scales: Sequence[torch.Tensor], act: str = "none",
                          bias_shards: Sequence[torch.Tensor | None] | None = None, out: str = "bf16",
                          y_shards: Sequence[torch.Tensor] | None = None,
                          y_scales: Sequence[torch.Tensor] | None = None, stream=None):
    """Y_r = act(X W_r^T + b_r) for every rank r on the 8-bit format, one launch.

    x and x_scales as tp_quantize_fp8 writes them (block_rows 1), each w_shards[r] and
    w_scales[r] with block_rows 128.  out="bf16" returns the list of Y_r; out="fp8" returns
    (codes, scales), two lists, ready for tp_linear_rowwise_fp8."""
    dev = _device_of("x", x)
    if out != "bf16" and out != "fp8":
        raise ValueError(f'out must be "bf16" or "fp8", got {out!r}')
    fp8 = out == "fp8"
    if not fp8 and y_scales is not None:
        raise ValueError('y_scales belongs to out="fp8"')
    p = _ranks(w_shards, w_scales, bias_shards, y_shards, y_scales)
    T, K = x.shape
    N = w_shards[0].shape[0]
    kg = _groups(K)
    ldx, ld_xs = _need("x", x, _E4M3, (T, K), dev), _need("x_scales", x_scales, _E8M0, (T, kg), dev)
    w, _ = _need_ranks("w_shards", w_shards, _E4M3, (N, K), dev, dense=True)
    ws, _ = _need_ranks("w_scales", w_scales, _E8M0, (_groups(N), kg), dev, dense=True)
    bias = None
    if bias_shards is not None:
        given = [b for b in bias_shards if b is not None]
        bias, _ = _need_ranks("bias_shards", given, _BF16, (N,), dev, dense=True)
        if len(given) != p:
            bias = _pointers[p](*[0 if b is None else b.data_ptr() for b in bias_shards])
    n = N // 2 if act == "swiglu" else N
    if y_shards is None:
        y_shards = _alloc(stream, x.device, _E4M3 if fp8 else _BF16, (T, n), p)
    y, ldy = _need_ranks("y_shards", y_shards, _E4M3 if fp8 else _BF16, (T, n), dev)
    ys, ld_ys = None, 0
    if fp8:
        s_shape = (T, _groups(n))
        if y_scales is None:
            y_scales = _alloc(stream, x.device, _E8M0, s_shape, p)
        ys, ld_ys = _need_ranks("y_scales", y_scales, _E8M0, s_shape, dev)
    _check(lib.tp_linear_colwise_fp8(x.data_ptr(), ldx, x_scales.data_ptr(), ld_xs, w, ws, bias, ACTS[act], p, T, K, N,
                                     y, ldy, ys, ld_ys, _launch_stream(stream, dev)))
    return (list(y_shards), list(y_scales)) if fp8 else list(y_shards)


def tp_linear_rowwise_fp8(x_shards: Sequence[torch.Tensor], x_scales: Sequence[torch.Tensor],
                          w_shards: Sequence[torch.Tensor], w_scales: Sequence[torch.Tensor],
                          bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Z = sum_r X_r W_r^T (+ bias once) on the 8-bit format, one launch; bf16 [T, N]."""
    p = _ranks(w_shards, w_scales, x_shards, x_scales)
    dev = _device_of("x_shards[0]", x_shards[0])
    T, K = x_shards[0].shape
    N = w_shards[0].shape[0]
    kg = _groups(K)
    w, _ = _need_ranks("w_shards", w_shards, _E4M3, (N, K), dev, dense=True)
    ws, _ = _need_ranks("w_scales", w_scales, _E8M0, (_groups(N), kg), dev, dense=True)
    x, ldx = _need_ranks("x_shards", x_shards, _E4M3, (T, K), dev)
    xs, ld_xs = _need_ranks("x_scales", x_scales, _E8M0, (T, kg), dev)
    if bias is not None:
        _need("bias", bias, _BF16, (N,), dev)
    if out is None:
        out, = _alloc(stream, x_shards[0].device, _BF16, (T, N))
    ldo = _need("out", out, _BF16, (T, N), dev)
    _check(lib.tp_linear_rowwise_fp8(x, ldx, xs, ld_xs, w, ws, None if bias is None else bias.data_ptr(), p, T, K, N,
                                     out.data_ptr(), ldo, _launch_stream(stream, dev)))
    return out


def tp_residual_norm(x: torch.Tensor, y: torch.Tensor | None = None, norm: str = "rms",
                     weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                     scale: torch.Tensor | None = None, shift: torch.Tensor | None = None, post_norm: str = "none",
                     post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
                     gate: torch.Tensor | None = None, alpha: float = 1.0, eps: float = 1e-6,
                     rows_per_mod: int | None = None, out: str | None = "bf16", h: torch.Tensor | None = None,
                     u: torch.Tensor | None = None, u_scales: torch.Tensor | None = None, stream=None):
    """h = alpha x + gate post_norm(y); u = norm(h) (1 + scale) + shift.  Returns (h, u, u_scales).

    gate, scale and shift are [D] vectors, used for every row of x, or [mod_rows, D] tables: row t
    uses table row t // rows_per_mod, which has to be given with more than one.  out: "bf16" or
    "fp8" (codes and scales), or None for h alone; what a call does not compute is returned as
    None.  Without a branch y there is no h."""
    dev = _device_of("x", x)
    if out not in ("bf16", "fp8", None):
        raise ValueError(f'out must be "bf16" or "fp8", got {out!r}')
    fp8 = out == "fp8"
    if u_scales is not None and not fp8:
        raise ValueError('u_scales belongs to out="fp8"')
    if u is not None and out is None:
        raise ValueError("u belongs to an output type")
    shape = x.shape
    T, D = shape
    ldx = 0 if x.dtype is _BF16 and x.is_contiguous() else _need("x", x, _BF16, shape, dev)

    vectors = [0, 0, 0, 0]
    if weight is not None or bias is not None or post_weight is not None or post_bias is not None:
        for i, (name, t) in enumerate((("weight", weight), ("bias", bias), ("post_weight", post_weight),
                                       ("post_bias", post_bias))):
            if t is not None:
                _need(name, t, _BF16, (D,), dev)
                vectors[i] = t.data_ptr()
    tables, mod = [0, 0, 0], None   # mod: (row stride, rows) of the tables
    if gate is not None or scale is not None or shift is not None:
        for i, (name, t) in enumerate((("gate", gate), ("scale", scale), ("shift", shift))):
            if t is not None:
                rows = 1 if t.dim() == 1 else t.shape[0]
                step = _need(name, t, _BF16, (D,) if t.dim() == 1 else (rows, D), dev)
                if mod is None:
                    mod = step, rows
                elif mod != (step, rows):
                    raise ValueError("gate, scale and shift must have the same rows and row stride")
                tables[i] = t.data_ptr()
        if rows_per_mod is None and mod[1] > 1:
            raise ValueError(f"tables of {mod[1]} rows need rows_per_mod, how many rows of x use each of them")
    y_at, ldy = 0, 0
    if y is not None:
        y_at, ldy = y.data_ptr(), _need("y", y, _BF16, shape, dev)
        if h is None:
            h, = _alloc(stream, x.device, _BF16, shape)
    h_at, ldh = (0, 0) if h is None else (h.data_ptr(), _need("h", h, _BF16, shape, dev))
    u_at, ldu, s_at, ld_us = 0, 0, 0, 0
    if out is not None:
        u_type = _E4M3 if fp8 else _BF16
        if u is None:
            u, = _alloc(stream, x.device, u_type, shape)
        u_at, ldu = u.data_ptr(), _need("u", u, u_type, shape, dev)
        if fp8:
            s_shape = (T, _groups(D))
            if u_scales is None:
                u_scales, = _alloc(stream, x.device, _E8M0, s_shape)
            s_at, ld_us = u_scales.data_ptr(), _need("u_scales", u_scales, _E8M0, s_shape, dev)
    ld_mod, mod_rows = mod or (0, 0)
    if mod and rows_per_mod is None:
        rows_per_mod = max(T, 1)
    args = _residual_norm_args(T, D, x.data_ptr(), ldx, y_at, ldy, NORMS[post_norm], vectors[2], vectors[3], alpha, eps,
                               *tables, ld_mod, mod_rows, rows_per_mod if mod else 0, h_at, ldh,
                               0 if out is None else NORMS[norm], vectors[0], vectors[1], u_at, ldu, s_at, ld_us)
    _check(lib.tp_residual_norm(args, _launch_stream(stream, dev)))
    return h, u, u_scales


# ---------------------------------------------------------------------------
# Paged 8-bit cache of keys and values
# ---------------------------------------------------------------------------

class PagedCache:
    """The keys and values of every rank's KV heads: tp_paged_cache (include/tp.h) over the caller's tensors.

    k[r] and v[r] are float8_e4m3fn [n_pages, n_kv_heads, page_size, head_dim], whole but for the
    stride from page to page; k_scales[r] and v_scales[r] are float8_e8m0fnu (or uint8) [n_pages,
    n_kv_heads].  The tensors are checked once, here, and kept: a program makes one cache for
    each layer and passes it to every call."""

    def __init__(self, k: Sequence[torch.Tensor], v: Sequence[torch.Tensor], k_scales: Sequence[torch.Tensor],
                 v_scales: Sequence[torch.Tensor]):
        n = len(k)
        if n < 1 or n > MAX_DEGREE:
            raise ValueError(f"k must have one entry for each of 1 to {MAX_DEGREE} ranks, got {n}")
        if not len(v) == len(k_scales) == len(v_scales) == n:
            raise ValueError(f"every list must have one entry for each of the {n} ranks")
        if k[0].dim() != 4:
            raise ValueError(f"k[0] must be [n_pages, n_kv_heads, page_size, head_dim], got {tuple(k[0].shape)}")
        shape = n_pages, heads, page, d = tuple(k[0].shape)
        self.device = k[0].device
        if not k[0].is_cuda:
            raise ValueError(f"k[0] must be on a CUDA device, got {k[0].device}")
        ld_page = self._strides("k and v", [*k, *v], (_E4M3,), shape, (page * d, d, 1))
        ld_scales = self._strides("k_scales and v_scales", [*k_scales, *v_scales], (_E8M0, _U8), (n_pages, heads), (1,))
        self.k, self.v, self.k_scales, self.v_scales = list(k), list(v), list(k_scales), list(v_scales)
        self.n_ranks, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n, n_pages, heads, page, d
        self._arrays = [_ptrs(ts) for ts in (k, v, k_scales, v_scales)]
        self._struct = _paged_cache(n, heads, d, page, n_pages, *[ctypes.addressof(a) for a in self._arrays], ld_page,
                                    ld_scales)

    @classmethod
    def empty(cls, n_ranks: int, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, device="cuda"):
        """A cache over new tensors (uninitialised: pages are read only where tokens were appended)."""
        codes = [[torch.empty((n_pages, n_kv_heads, page_size, head_dim), dtype=_E4M3, device=device)
                  for _ in range(n_ranks)] for _ in range(2)]
        scales = [[torch.empty((n_pages, n_kv_heads), dtype=_E8M0, device=device) for _ in range(n_ranks)]
                  for _ in range(2)]
        return cls(*codes, *scales)

    def _strides(self, name, ts, dtypes, shape, inner) -> int:
        """The stride from page to page (0: whole tensors), the same for every tensor."""
        steps = set()
        for t in ts:
            if t.dtype not in dtypes:
                raise TypeError(f"{name} must be {dtypes[0]}, got {t.dtype}")
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must all have the shape {shape}, got {tuple(t.shape)}")
            if t.device != self.device:
                raise ValueError(f"{name} must all be on {self.device}, got {t.device}")
            if t.is_contiguous():
                steps.add(shape[1] * inner[0] if len(inner) > 1 else shape[1])
                continue
            if any(size > 1 and got != want for size, got, want in zip(shape[1:], t.stride()[1:], inner)):
                raise ValueError(f"{name} must be whole but for the stride from page to page, got strides {t.stride()}")
            if t.stride(0) < shape[1] * inner[0]:
                raise ValueError(f"{name}: a stride of {t.stride(0)} overlaps pages of {shape[1] * inner[0]} elements")
            steps.add(t.stride(0))
        if len(steps) > 1:
            raise ValueError(f"{name} must all have the same stride from page to page")
        return steps.pop()


class PagedBatch:
    """The sequences of a step and where their tokens are: tp_paged_batch (include/tp.h) over int32 tensors on the GPU.

    seq_start [n_seqs + 1], kv_len [n_seqs] and page_table [n_seqs, max_pages] are read when the
    kernels run; max_new (or max_q, its other name: the rows of Q) is at least the new rows of any
    sequence.  Made once a step, for every layer."""

    def __init__(self, seq_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor,
                 max_new: int | None = None, max_q: int | None = None):
        if (max_new is None) == (max_q is None):
            raise TypeError("one of max_new and max_q, its other name, is needed")
        max_new = max_q if max_new is None else max_new
        if page_table.dim() != 2:
            raise ValueError(f"page_table must be [n_seqs, max_pages], got {tuple(page_table.shape)}")
        n, max_pages = page_table.shape
        self.device = page_table.device
        if not page_table.is_cuda:
            raise ValueError(f"page_table must be on a CUDA device, got {page_table.device}")
        for name, t, shape in (("seq_start", seq_start, (n + 1,)), ("kv_len", kv_len, (n,)),
                               ("page_table", page_table, (n, max_pages))):
            if t.dtype is not torch.int32:
                raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
        ld = [_need(name, t, torch.int32, torch.Size(shape), page_table.get_device())
              for name, t, shape in (("seq_start", seq_start, (n + 1,)), ("kv_len", kv_len, (n,)),
                                     ("page_table", page_table, (n, max_pages)))][2]
        self.seq_start, self.kv_len, self.page_table = seq_start, kv_len, page_table
        if not 0 <= max_new < 2 ** 31:
            raise ValueError(f"max_new must be in 0 .. 2**31 - 1, got {max_new}")
        self.n_seqs, self.max_pages, self.max_new = n, max_pages, int(max_new)
        self._struct = _paged_batch(n, self.max_new, seq_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), ld,
                                    max_pages)


def _paged_device(cache: PagedCache, batch: PagedBatch) -> int:
    dev = cache.device.index
    if dev != torch._C._cuda_getDevice() or batch.device.index != dev:
        raise ValueError(f"cache ({cache.device}) and batch ({batch.device}) must be on the current CUDA device")
    return dev


def tp_kv_append_fp8(qkv: Sequence[torch.Tensor], n_heads: int, cache: PagedCache, batch: PagedBatch,
                     rope: str | None = None, cos_sin: torch.Tensor | None = None,
                     positions: torch.Tensor | None = None, q_out: Sequence[torch.Tensor] | None = None,
                     stream=None) -> list[torch.Tensor]:
    """Every rank's new keys (rotated) and values into its cache, one launch; returns each rank's Q, rotated.

    qkv[r] is bf16 [T, (n_heads + 2 n_kv_heads) head_dim], rank r's colwise Q, K and V columns.
    rope names the pairs of the rotation, "half" or "pairs"; cos_sin is then its fp32 table
    [n_positions, rot_dim], cosines before sines, and positions (int32 [T]) the table row of each
    token (default: its position in the cache).  q_out[r] may be qkv[r][:, :n_heads * head_dim]."""
    dev = _paged_device(cache, batch)
    n = cache.n_ranks
    if len(qkv) != n or (q_out is not None and len(q_out) != n):
        raise ValueError(f"qkv and q_out must have one entry for each of the cache's {n} ranks")
    if qkv[0].dim() != 2:
        raise ValueError(f"qkv[0] must be 2-D, got {tuple(qkv[0].shape)}")
    T, wide = qkv[0].shape[0], n_heads * cache.head_dim
    at, ld = _need_ranks("qkv", qkv, _BF16, (T, wide + 2 * cache.n_kv_heads * cache.head_dim), dev)
    turn = None
    if rope is not None:
        if rope not in ROPE_STYLES:
            raise ValueError(f'rope must be "half" or "pairs", got {rope!r}')
        if cos_sin is None or cos_sin.dim() != 2:
            raise ValueError("a rotation needs cos_sin, [n_positions, rot_dim]")
        step = _need("cos_sin", cos_sin, torch.float32, cos_sin.shape, dev)
        if positions is not None:
            _need("positions", positions, torch.int32, (T,), dev)
        turn = _rope(ROPE_STYLES[rope], cos_sin.shape[1], cos_sin.data_ptr(), step, cos_sin.shape[0],
                     0 if positions is None else positions.data_ptr())
    elif cos_sin is not None or positions is not None:
        raise ValueError('cos_sin and positions belong to rope="half" or rope="pairs"')
    if n_heads == 0:
        q_out, q_at, ld_q = [], None, 0
    else:
        if q_out is None:
            q_out = _alloc(stream, cache.device, _BF16, (T, wide), n)
        q_at, ld_q = _need_ranks("q_out", q_out, _BF16, (T, wide), dev)
    _check(lib.tp_kv_append_fp8(cache._struct, batch._struct, at, ld, T, n_heads, turn, q_at, ld_q,
                                _launch_stream(stream, dev)))
    return list(q_out)


def tp_attention_paged_workspace_bytes(cache: PagedCache, batch: PagedBatch, T: int, n_heads: int) -> int:
    return int(lib.tp_attention_paged_workspace_bytes(cache._struct, batch._struct, T, n_heads))


def tp_attention_paged_fp8(q: Sequence[torch.Tensor], cache: PagedCache, batch: PagedBatch, scale: float | None = None,
                           causal: bool = True, window: int = 0, outs: Sequence[torch.Tensor] | None = None,
                           workspace: torch.Tensor | None = None, stream=None) -> list[torch.Tensor]:
    """softmax(scale Q_h K_g^T) V_g of every rank's new tokens over its cache, g the KV head of query head h.

    q[r] is bf16 [T, n_heads * head_dim]; scale defaults to head_dim ** -0.5.  A token sees the
    keys of its sequence up to its own position (causal), the last `window` of them where window > 0."""
    dev = _paged_device(cache, batch)
    n, d = cache.n_ranks, cache.head_dim
    if len(q) != n or (outs is not None and len(outs) != n):
        raise ValueError(f"q and outs must have one entry for each of the cache's {n} ranks")
    shape = q[0].shape
    if len(shape) != 2 or shape[1] % d != 0:
        raise ValueError(f"q[0] must be [T, n_heads * {d}], got {tuple(shape)}")
    T, n_heads = shape[0], shape[1] // d
    at, ld = _need_ranks("q", q, _BF16, shape, dev)
    if outs is None:
        outs = _alloc(stream, cache.device, _BF16, shape, n)
    out_at, ldo = _need_ranks("outs", outs, _BF16, shape, dev)
    if workspace is None:
        need = tp_attention_paged_workspace_bytes(cache, batch, T, n_heads)
        if need:
            workspace, = _alloc(stream, cache.device, _U8, (need,))
    ws_at, ws_bytes = 0, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the current CUDA device")
        ws_at, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib.tp_attention_paged_fp8(cache._struct, batch._struct, at, ld, T, n_heads,
                                      d ** -0.5 if scale is None else scale, int(causal), min(window, 2 ** 31 - 1), ws_at, ws_bytes, out_at,
                                      ldo, _launch_stream(stream, dev)))
    return list(outs)


# ---------------------------------------------------------------------------
# Diagnostics
# ---------------------------------------------------------------------------

def tp_last_error() -> str:
    return lib.tp_last_error().decode()


def tp_status_name(status: int) -> str:
    return lib.tp_status_name(status).decode()


def tp_device_status(stream=None) -> None:
    """Synchronise the stream; raise TPError if a kernel gave up on a bounded wait or met a bad index (paged cache)."""
    _check(lib.tp_device_status(_stream(stream)))


def tp_abi_version() -> int:
    return int(lib.tp_abi_version())


def tp_set_tile_wait_limit_ns(ns: int) -> None:
    """Bound, in ns, on a workspace-mode CTA's wait for the other ranks' partials (0: the default 2 s)."""
    lib.tp_set_tile_wait_limit_ns(int(ns))


def tp_tile_wait_limit_ns() -> int:
    return int(lib.tp_tile_wait_limit_ns())


def bf16_from_bits(bits, device=None) -> torch.Tensor:
    """A bf16 tensor holding the given uint16 bit patterns (numpy array), optionally moved to `device`."""
    import numpy as np
    t = torch.from_numpy(np.ascontiguousarray(bits, dtype=np.uint16).view(np.int16)).view(torch.bfloat16)
    return t.to(device) if device is not None else t


def bits_from_bf16(t: torch.Tensor):
    """uint16 numpy bit patterns of a bf16 tensor (copied to the host)."""
    import numpy as np
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


# ---------------------------------------------------------------------------
# Shard-on-read from a safetensors file (include/tp_safetensors.h)
# ---------------------------------------------------------------------------

ST_DTYPES = ["BOOL", "U8", "I8", "F8_E4M3", "F8_E5M2", "I16", "U16", "F16", "BF16", "I32", "U32", "F32", "I64",
             "U64", "F64"]
ST_MAX_DIMS = 8
_ST_TORCH = {"BOOL": "bool", "U8": "uint8", "I8": "int8", "F8_E4M3": "float8_e4m3fn", "F8_E5M2": "float8_e5m2",
             "I16": "int16", "U16": "uint16", "F16": "float16", "BF16": "bfloat16", "I32": "int32", "U32": "uint32",
             "F32": "float32", "I64": "int64", "U64": "uint64", "F64": "float64"}


def st_torch_dtype(dtype: str) -> torch.dtype:
    """The torch dtype holding a safetensors dtype's elements."""
    return getattr(torch, _ST_TORCH[dtype])


def tp_st_dtype_size(dtype: str) -> int:
    return int(lib.tp_st_dtype_size(ST_DTYPES.index(dtype)))


def tp_st_open(path: str, staging_bytes: int = 0) -> int:
    """Open a safetensors file and check its header; returns the handle (close it with tp_st_close)."""
    h = _vp()
    _check(lib.tp_st_open(os.fsencode(path), staging_bytes, ctypes.byref(h)))
    return h.value


def tp_st_close(handle: int) -> None:
    _check(lib.tp_st_close(handle))


ST_READ_MODES = ["auto", "staged", "mapped"]   # tp_st_read_mode order


def tp_st_set_read_mode(handle: int, mode: str) -> None:
    """How the following loads read the file: "auto", "staged" or "mapped"."""
    _check(lib.tp_st_set_read_mode(handle, ST_READ_MODES.index(mode)))


def tp_st_read_mode_on_device(handle: int) -> str:
    """The mode a load on the current device uses ("staged" or "mapped")."""
    m = ctypes.c_int(-1)
    _check(lib.tp_st_read_mode_on_device(handle, ctypes.byref(m)))
    return ST_READ_MODES[m.value]


def tp_st_count(handle: int) -> int:
    return int(lib.tp_st_count(handle))


def tp_st_info(handle: int, index: int) -> dict:
    name = ctypes.c_char_p()
    dtype, ndim = ctypes.c_int(), ctypes.c_int()
    shape = (_i64 * ST_MAX_DIMS)()
    off, nbytes = ctypes.c_uint64(), ctypes.c_uint64()
    _check(lib.tp_st_info(handle, index, ctypes.byref(name), ctypes.byref(dtype), ctypes.byref(ndim), shape,
                          ctypes.byref(off), ctypes.byref(nbytes)))
    return {"name": name.value.decode("utf-8"), "dtype": ST_DTYPES[dtype.value],
            "shape": tuple(shape[i] for i in range(ndim.value)), "offset": off.value, "nbytes": nbytes.value}


def tp_st_find(handle: int, name: str) -> int:
    return int(lib.tp_st_find(handle, name.encode("utf-8")))


def _st_shard_shape(info: dict, style: str, tp_degree: int) -> tuple:
    shape = info["shape"]
    if style == "colwise":
        if not shape:
            return ()
        return (shape[0] // tp_degree, *shape[1:])
    return (shape[0], shape[1] // tp_degree) if len(shape) == 2 else shape


def tp_st_plan_shard_ranks(handle: int, name: str, style: str, tp_degree: int, rank_begin: int = 0,
                           rank_count: int | None = None, fused_splits: Sequence[int] | None = None,
                           num_heads: int = 0, head_dim: int = 0, outs: Sequence[torch.Tensor] | None = None,
                           device=None, stream=None) -> list[torch.Tensor]:
    """Ranks [rank_begin, rank_begin + rank_count)'s shards of tensor ``name``, read from the file to the GPU."""
    if rank_count is None:
        rank_count = tp_degree - rank_begin
    arr, n = _splits(fused_splits)
    if outs is None:
        idx = tp_st_find(handle, name)
        if idx < 0:
            raise TPError(STATUS_NAMES.index("TP_ERR_NOT_FOUND"), f"TP_ERR_NOT_FOUND: no tensor {name!r}")
        info = tp_st_info(handle, idx)
        # Validate before allocating: a refused plan allocates nothing.
        _check(lib.tp_st_plan_shard_ranks(handle, name.encode("utf-8"), STYLES[style], tp_degree, rank_begin, 0, arr,
                                          n, num_heads, head_dim, None, None))
        dev = device if device is not None else torch.device("cuda")
        outs = [torch.empty(_st_shard_shape(info, style, tp_degree), dtype=st_torch_dtype(info["dtype"]), device=dev)
                for _ in range(rank_count)]
    _check(lib.tp_st_plan_shard_ranks(handle, name.encode("utf-8"), STYLES[style], tp_degree, rank_begin, rank_count,
                                      arr, n, num_heads, head_dim, _ptrs(outs) if outs else None, _stream(stream)))
    return list(outs)


class SafetensorsFile:
    """A safetensors file opened for shard-on-read (closes on exit of a ``with`` block)."""

    def __init__(self, path: str, staging_bytes: int = 0, read_mode: str = "auto"):
        self.handle = tp_st_open(path, staging_bytes)
        if read_mode != "auto":
            try:
                tp_st_set_read_mode(self.handle, read_mode)
            except BaseException:
                self.close()
                raise

    def read_mode_on_device(self) -> str:
        return tp_st_read_mode_on_device(self.handle)

    def tensors(self) -> list[dict]:
        return [tp_st_info(self.handle, i) for i in range(tp_st_count(self.handle))]

    def shard_ranks(self, name: str, style: str, tp_degree: int, **kw) -> list[torch.Tensor]:
        return tp_st_plan_shard_ranks(self.handle, name, style, tp_degree, **kw)

    def close(self) -> None:
        if self.handle:
            h, self.handle = self.handle, None
            tp_st_close(h)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
