"""ctypes binding of libmoe.so.

Argument marshalling only: every step of the layer runs in the HIP library.
PyTorch supplies device memory and the stream; nothing here computes.  If
the library is missing, loading raises -- there is no fallback.

The functions carry the C names (see include/moe.h for the operations,
layouts and error codes).  Output tensors may be passed in (to reuse
buffers, e.g. under graph capture) or are allocated on the input's device.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")
_lib = None

MOE_ACT_GELU = 0
MOE_ACT_SWIGLU = 1
ACTS = {"gelu": MOE_ACT_GELU, "swiglu": MOE_ACT_SWIGLU}
MOE_ACT_NONE = 2
MOE_ACT_SILU = 3
LINEAR_ACTS = {**ACTS, "none": MOE_ACT_NONE, "silu": MOE_ACT_SILU}
SCORES = {"softmax": 0, "sigmoid": 1}
OUT_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f32 = ctypes.c_float

_SIGNATURES = {
    "moe_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_abi_version": (_i32, []),
    "moe_rows_capacity": (_i64, [_i64, _i32, _i32, _i32]),
    "moe_tiles_capacity": (_i64, [_i64, _i32, _i32, _i32]),
    "moe_permute_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32]),
    "moe_grouped_ffn_workspace_bytes": (_sz, [_i32, _i32]),
    "moe_route_topk": (ctypes.c_int, [_p, _i64, _i32, _i32, _i32, _p, _p, _p]),
    "moe_permute": (ctypes.c_int, [_p, _p, _p, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                   _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "moe_permute_noalloc": (ctypes.c_int, [_p, _p, _p, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                           _p, _p, _p, _p, _p, _p, _p, _p]),
    "moe_grouped_ffn": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32,
                                       _i64, _i64, _p, _p, _p, _sz, _p]),
    "moe_grouped_ffn_gather": (ctypes.c_int, [_p, _p, _i64, _i32, _p, _p, _p, _p, _p, _p, _p, _i32, _i32, _i32,
                                              _i32, _i32, _i64, _i64, _p, _p, _p, _sz, _p]),
    "moe_ffn_combine_fused_workspace_bytes": (_sz, [_i64, _i32]),
    "moe_ffn_combine_fused": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _i64, _i64,
                                             _p, _p, _p, _p, _i64, _i32, _p, _p, _sz, _p]),
    "moe_combine": (ctypes.c_int, [_p, _p, _p, _i64, _i32, _i32, _i64, _p, _p]),
    "moe_route_grouped": (ctypes.c_int, [_p, _p, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _p, _p, _p]),
    "moe_route_grouped_backward": (ctypes.c_int, [_p, _p, _p, _i64, _i32, _i32, _i32, _i32, _f32, _p, _p]),
    "moe_route_grouped_bias_backward": (ctypes.c_int, [_p, _p, _p, _p, _i64, _i32, _i32, _i32, _i32, _f32, _p, _p]),
    "moe_combine_backward": (ctypes.c_int, [_p, _p, _p, _p, _i64, _i32, _i32, _i64, _p, _p, _p]),
    "moe_linear_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32]),
    "moe_linear": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i32, _i32, _i32, _i32, _p, _p, _p, _p, _sz, _p]),
    "moe_linear_backward_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32]),
    "moe_linear_backward": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i32, _i32, _i32, _i32, _p, _p, _p, _p, _p,
                                           _p, _sz, _p]),
}


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {lib().moe_status_str(status).decode()} ({status})")


def lib_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built by mixture_experts_layer_moe_amd.build); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: build it with "
                              "`python -m mixture_experts_layer_moe_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status)


def _need(t: torch.Tensor, dtype, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def rows_capacity(T: int, k: int, E_loc: int, tile_m: int) -> int:
    return int(lib().moe_rows_capacity(T, k, E_loc, tile_m))


def tiles_capacity(T: int, k: int, E_loc: int, tile_m: int) -> int:
    return int(lib().moe_tiles_capacity(T, k, E_loc, tile_m))


def permute_workspace_bytes(T: int, k: int, E_loc: int, num_ranks: int) -> int:
    return int(lib().moe_permute_workspace_bytes(T, k, E_loc, num_ranks))


def grouped_ffn_workspace_bytes(tile_m: int, H: int) -> int:
    return int(lib().moe_grouped_ffn_workspace_bytes(tile_m, H))


# ---------------------------------------------------------------------------
# the four calls
# ---------------------------------------------------------------------------

def moe_route_topk(logits: torch.Tensor, k: int, renormalize: bool = True,
                   topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                   stream=None):
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    dev = logits.device
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
    _check("moe_route_topk", lib().moe_route_topk(_ptr(logits), T, E, k, int(bool(renormalize)),
                                                  _ptr(topk_idx), _ptr(topk_w), _stream(stream)))
    return topk_idx, topk_w


@dataclass
class Permuted:
    """Outputs of moe_permute (all device tensors; counts stay on the device)."""
    x_perm: Optional[torch.Tensor]  # [R_cap, H] bf16, or None for an index-only permute
    expert_counts: torch.Tensor   # [E_loc] int32
    expert_offsets: torch.Tensor  # [E_loc + 1] int32
    row_src: torch.Tensor         # [R_cap] int32
    inv_perm: torch.Tensor        # [T, k] int32
    tiles: torch.Tensor           # [tiles_cap, 2] int32
    num_tiles: torch.Tensor       # [1] int32
    tile_m: int
    R_cap: int
    tiles_cap: int


def alloc_permuted(T: int, H: int, k: int, E_loc: int, tile_m: int, device, rows: bool = True) -> Permuted:
    """Outputs for moe_permute; rows=False leaves out x_perm (index-only permute)."""
    R_cap = rows_capacity(T, k, E_loc, tile_m)
    tcap = tiles_capacity(T, k, E_loc, tile_m)
    i32 = dict(dtype=torch.int32, device=device)
    return Permuted(
        x_perm=torch.empty((R_cap, H), dtype=torch.bfloat16, device=device) if rows else None,
        expert_counts=torch.empty(E_loc, **i32), expert_offsets=torch.empty(E_loc + 1, **i32),
        row_src=torch.empty(R_cap, **i32), inv_perm=torch.empty((T, k), **i32),
        tiles=torch.empty((tcap, 2), **i32), num_tiles=torch.empty(1, **i32),
        tile_m=tile_m, R_cap=R_cap, tiles_cap=tcap)


def moe_permute(x: torch.Tensor, topk_idx: torch.Tensor, src_rank: Optional[torch.Tensor], E: int,
                expert_begin: int, E_loc: int, num_ranks: int, tile_m: int,
                out: Optional[Permuted] = None, ws: Optional[torch.Tensor] = None,
                stream=None, copy_rows: bool = True) -> Permuted:
    """copy_rows=False writes only the indices (for moe_grouped_ffn_gather)."""
    _need(x, torch.bfloat16, "x")
    _need(topk_idx, torch.int32, "topk_idx")
    if src_rank is not None:
        _need(src_rank, torch.int32, "src_rank")
    T, H = x.shape
    k = topk_idx.shape[1]
    if out is None:
        out = alloc_permuted(T, H, k, E_loc, tile_m, x.device, rows=copy_rows)
    copy_rows = copy_rows and out.x_perm is not None
    nbytes = permute_workspace_bytes(T, k, E_loc, num_ranks)
    if ws is None:
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _check("moe_permute", lib().moe_permute(
        _ptr(x) if copy_rows else None, _ptr(topk_idx), _ptr(src_rank), T, H, k, E, expert_begin, E_loc, num_ranks, tile_m,
        _ptr(out.x_perm) if copy_rows else None, _ptr(out.expert_counts), _ptr(out.expert_offsets),
        _ptr(out.row_src),
        _ptr(out.inv_perm), _ptr(out.tiles), _ptr(out.num_tiles), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def moe_permute_noalloc(x: Optional[torch.Tensor], topk_idx: torch.Tensor, src_rank: Optional[torch.Tensor],
                        H: int, E: int, expert_begin: int, E_loc: int, num_ranks: int, tile_m: int,
                        out: Permuted, stream=None) -> int:
    """moe_permute on the library's fixed scratch, into preallocated outputs; returns the status code.

    x may be None (with out.x_perm None) for an index-only permute.  Nothing is
    allocated here: the caller passes every output.
    """
    _need(topk_idx, torch.int32, "topk_idx")
    if src_rank is not None:
        _need(src_rank, torch.int32, "src_rank")
    T, k = topk_idx.shape
    return int(lib().moe_permute_noalloc(
        _ptr(x), _ptr(topk_idx), _ptr(src_rank), T, H, k, E, expert_begin, E_loc, num_ranks, tile_m,
        _ptr(out.x_perm), _ptr(out.expert_counts), _ptr(out.expert_offsets), _ptr(out.row_src),
        _ptr(out.inv_perm), _ptr(out.tiles), _ptr(out.num_tiles), _stream(stream)))


def moe_grouped_ffn(p: Permuted, w0: torch.Tensor, w0_up: Optional[torch.Tensor], w1: torch.Tensor,
                    act: str, act_buf: Optional[torch.Tensor] = None,
                    y_perm: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None, use_workspace: bool = True):
    _need(w0, torch.bfloat16, "w0")
    _need(w1, torch.bfloat16, "w1")
    if w0_up is not None:
        _need(w0_up, torch.bfloat16, "w0_up")
    E_loc, F, H = w0.shape
    dev = w0.device
    if act_buf is None:
        act_buf = torch.empty((p.R_cap, F), dtype=torch.bfloat16, device=dev)
    if y_perm is None:
        y_perm = torch.empty((p.R_cap, H), dtype=torch.float32, device=dev)
    if ws is None and use_workspace:
        nbytes = grouped_ffn_workspace_bytes(p.tile_m, H)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _check("moe_grouped_ffn", lib().moe_grouped_ffn(
        _ptr(p.x_perm), _ptr(p.expert_counts), _ptr(p.expert_offsets), _ptr(p.tiles), _ptr(p.num_tiles),
        _ptr(w0), _ptr(w0_up), _ptr(w1), E_loc, H, F, ACTS[act], p.tile_m, p.R_cap, p.tiles_cap,
        _ptr(act_buf), _ptr(y_perm), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return act_buf, y_perm


def moe_grouped_ffn_gather(x: torch.Tensor, p: Permuted, w0: torch.Tensor, w0_up: Optional[torch.Tensor],
                           w1: torch.Tensor, act: str, act_buf: Optional[torch.Tensor] = None,
                           y_perm: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                           stream=None, use_workspace: bool = True):
    """moe_grouped_ffn with layer0 reading its rows from x through p.row_src (no x_perm needed)."""
    _need(x, torch.bfloat16, "x")
    _need(w0, torch.bfloat16, "w0")
    _need(w1, torch.bfloat16, "w1")
    if w0_up is not None:
        _need(w0_up, torch.bfloat16, "w0_up")
    T, k = p.inv_perm.shape
    E_loc, F, H = w0.shape
    dev = w0.device
    if act_buf is None:
        act_buf = torch.empty((p.R_cap, F), dtype=torch.bfloat16, device=dev)
    if y_perm is None:
        y_perm = torch.empty((p.R_cap, H), dtype=torch.float32, device=dev)
    if ws is None and use_workspace:
        nbytes = grouped_ffn_workspace_bytes(p.tile_m, H)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _check("moe_grouped_ffn_gather", lib().moe_grouped_ffn_gather(
        _ptr(x), _ptr(p.row_src), T, k, _ptr(p.expert_counts), _ptr(p.expert_offsets), _ptr(p.tiles),
        _ptr(p.num_tiles), _ptr(w0), _ptr(w0_up), _ptr(w1), E_loc, H, F, ACTS[act], p.tile_m, p.R_cap,
        p.tiles_cap, _ptr(act_buf), _ptr(y_perm), _ptr(ws), 0 if ws is None else ws.numel(),
        _stream(stream)))
    return act_buf, y_perm


def fused_workspace_bytes(tiles_cap: int, H: int) -> int:
    return int(lib().moe_ffn_combine_fused_workspace_bytes(tiles_cap, H))


def alloc_fused_workspace(tiles_cap: int, H: int, device) -> torch.Tensor:
    """Zero-filled workspace of moe_ffn_combine_fused (each launch leaves it zero again)."""
    nbytes = fused_workspace_bytes(tiles_cap, H)
    if nbytes == 0:
        raise ValueError("moe_ffn_combine_fused does not support this shape")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def fused_error_word(ws: torch.Tensor) -> int:
    """The fused launch's error word (nonzero: a wait timed out; the caller clears it)."""
    return int(ws[:4].view(torch.int32).item())


def moe_ffn_combine_fused(p: Permuted, w0: torch.Tensor, w0_up: Optional[torch.Tensor], w1: torch.Tensor,
                          act: str, topk_w: torch.Tensor, ws: torch.Tensor,
                          act_buf: Optional[torch.Tensor] = None, y_perm: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, stream=None):
    """Grouped FFN and combine as one launch with tile-level signals; returns (act_buf, y_perm, out)."""
    _need(w0, torch.bfloat16, "w0")
    _need(w1, torch.bfloat16, "w1")
    _need(topk_w, torch.float32, "topk_w")
    if w0_up is not None:
        _need(w0_up, torch.bfloat16, "w0_up")
    E_loc, F, H = w0.shape
    T, k = p.inv_perm.shape
    dev = w0.device
    if act_buf is None:
        act_buf = torch.empty((p.R_cap, F), dtype=torch.bfloat16, device=dev)
    if y_perm is None:
        y_perm = torch.empty((p.R_cap, H), dtype=torch.float32, device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=dev)
    _check("moe_ffn_combine_fused", lib().moe_ffn_combine_fused(
        _ptr(p.x_perm), _ptr(p.expert_counts), _ptr(p.expert_offsets), _ptr(p.tiles), _ptr(p.num_tiles),
        _ptr(w0), _ptr(w0_up), _ptr(w1), E_loc, H, F, ACTS[act], p.tile_m, p.R_cap, p.tiles_cap,
        _ptr(act_buf), _ptr(y_perm), _ptr(p.inv_perm), _ptr(topk_w), T, k, _ptr(out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return act_buf, y_perm, out


def moe_combine(y_perm: torch.Tensor, inv_perm: torch.Tensor, topk_w: torch.Tensor,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _need(y_perm, torch.float32, "y_perm")
    _need(inv_perm, torch.int32, "inv_perm")
    _need(topk_w, torch.float32, "topk_w")
    T, k = inv_perm.shape
    R_cap, H = y_perm.shape
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=y_perm.device)
    _check("moe_combine", lib().moe_combine(_ptr(y_perm), _ptr(inv_perm), _ptr(topk_w), T, k, H, R_cap,
                                            _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# Operators beside the path: grouped routing, dense projection, gradients.
#
# These check every tensor (type, shape, contiguity, one device for all) and
# launch on the tensors' device, whichever device is current.
# ---------------------------------------------------------------------------

def _take(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int, optional: bool = False):
    """Address of a checked argument on device number `dev` (None for an absent optional one)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _matrix(t: torch.Tensor, name: str):
    """(rows, columns) of a two-dimensional argument."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    return t.shape


def _launch(fn, name: str, dev: int, *args):
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise MoEError(name, status)


def _on(stream, call, *args, **kw):
    """The call with `stream` current, so that its allocations belong to that stream as its launches do."""
    for t in (*args, *kw.values()):
        if isinstance(t, torch.Tensor) and t.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, a tensor on {t.device}")
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _choice(table: dict, key, name: str) -> int:
    if key not in table:
        raise ValueError(f"{name} must be one of {sorted(map(str, table))}, got {key!r}")
    return table[key]


def moe_route_grouped(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None, score: str = "softmax",
                      n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                      scale: float = 1.0, topk_idx: Optional[torch.Tensor] = None,
                      topk_w: Optional[torch.Tensor] = None, stream=None):
    """Top-k routing by score + bias inside the best groups; returns (topk_idx, topk_w)."""
    if stream is not None:
        return _on(stream, moe_route_grouped, logits, k, bias, score, n_group, topk_group, group_top, renormalize, scale,
                   topk_idx, topk_w)
    T, E = _matrix(logits, "logits")
    dev = logits.get_device()
    if topk_idx is None:
        topk_idx = torch.empty((T, max(k, 0)), dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty((T, max(k, 0)), dtype=torch.float32, device=logits.device)
    f32 = torch.float32
    _launch((_lib or lib()).moe_route_grouped, "moe_route_grouped", dev, _take(logits, "logits", f32, (T, E), dev),
            _take(bias, "bias", f32, (E,), dev, True), T, E, k, _choice(SCORES, score, "score"), n_group, topk_group,
            group_top, 1 if renormalize else 0, scale, _take(topk_idx, "topk_idx", torch.int32, (T, k), dev),
            _take(topk_w, "topk_w", f32, (T, k), dev))
    return topk_idx, topk_w


def moe_route_grouped_backward(logits: torch.Tensor, topk_idx: torch.Tensor, d_topk_w: torch.Tensor,
                               score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                               d_logits: Optional[torch.Tensor] = None, stream=None,
                               bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of moe_route_grouped's topk_w with respect to logits, for its choice topk_idx; bias: the forward call's,
    which matters where it bars experts (-inf or NaN)."""
    if stream is not None:
        return _on(stream, moe_route_grouped_backward, logits, topk_idx, d_topk_w, score, renormalize, scale, d_logits,
                   bias=bias)
    T, E = _matrix(logits, "logits")
    dev, k = logits.get_device(), _matrix(topk_idx, "topk_idx")[1]
    if d_logits is None:
        d_logits = torch.empty_like(logits)
    f32 = torch.float32
    _launch((_lib or lib()).moe_route_grouped_bias_backward, "moe_route_grouped_backward", dev,
            _take(logits, "logits", f32, (T, E), dev), _take(bias, "bias", f32, (E,), dev, True), _take(topk_idx, "topk_idx", torch.int32, (T, k), dev),
            _take(d_topk_w, "d_topk_w", f32, (T, k), dev), T, E, k, _choice(SCORES, score, "score"),
            1 if renormalize else 0, scale, _take(d_logits, "d_logits", f32, (T, E), dev))
    return d_logits


def moe_combine_backward(d_out: torch.Tensor, y_perm: torch.Tensor, inv_perm: torch.Tensor, topk_w: torch.Tensor,
                         d_y_perm: Optional[torch.Tensor] = None, d_topk_w: Optional[torch.Tensor] = None, stream=None):
    """Gradients of moe_combine: (d_y_perm, d_topk_w); rows of d_y_perm that no slot names are left as they were."""
    if stream is not None:
        return _on(stream, moe_combine_backward, d_out, y_perm, inv_perm, topk_w, d_y_perm, d_topk_w)
    T, H = _matrix(d_out, "d_out")
    dev, R_cap, k = d_out.get_device(), _matrix(y_perm, "y_perm")[0], _matrix(inv_perm, "inv_perm")[1]
    if d_y_perm is None:
        d_y_perm = torch.empty_like(y_perm)
    if d_topk_w is None:
        d_topk_w = torch.empty((T, k), dtype=torch.float32, device=d_out.device)
    f32 = torch.float32
    _launch((_lib or lib()).moe_combine_backward, "moe_combine_backward", dev, _take(d_out, "d_out", f32, (T, H), dev),
            _take(y_perm, "y_perm", f32, (R_cap, H), dev), _take(inv_perm, "inv_perm", torch.int32, (T, k), dev),
            _take(topk_w, "topk_w", f32, (T, k), dev), T, k, H, R_cap, _take(d_y_perm, "d_y_perm", f32, (R_cap, H), dev),
            _take(d_topk_w, "d_topk_w", f32, (T, k), dev))
    return d_y_perm, d_topk_w


def linear_workspace_bytes(M: int, N: int, K: int, act: str) -> int:
    return int(lib().moe_linear_workspace_bytes(M, N, K, _choice(LINEAR_ACTS, act, "act")))


def linear_backward_workspace_bytes(M: int, N: int, K: int, act: str) -> int:
    return int(lib().moe_linear_backward_workspace_bytes(M, N, K, _choice(LINEAR_ACTS, act, "act")))


def _alloc_ws(nbytes: int, device) -> Optional[torch.Tensor]:
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def alloc_linear_workspace(M: int, N: int, K: int, act: str, device) -> Optional[torch.Tensor]:
    """Workspace of moe_linear on that device (None where this size needs none)."""
    with torch.cuda.device(device):
        return _alloc_ws(linear_workspace_bytes(M, N, K, act), device)


def alloc_linear_backward_workspace(M: int, N: int, K: int, act: str, device) -> Optional[torch.Tensor]:
    """Workspace of moe_linear_backward on that device (None for no rows)."""
    with torch.cuda.device(device):
        return _alloc_ws(linear_backward_workspace_bytes(M, N, K, act), device)


def _ws(ws: Optional[torch.Tensor], dev: int):
    if ws is None:
        return None, 0
    n = ws.numel()
    return _take(ws, "ws", torch.uint8, (n,), dev), n


def moe_linear(x: torch.Tensor, w: torch.Tensor, w_up: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, bias_up: Optional[torch.Tensor] = None, act: str = "none",
               residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, z: Optional[torch.Tensor] = None,
               z_up: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None,
               use_workspace: bool = True) -> torch.Tensor:
    """act(x . w^T + bias) (SwiGLU: silu(.) * (x . w_up^T + bias_up)) + residual; z, z_up: buffers for the
    pre-activations that moe_linear_backward needs.  out may be residual itself; its type wins over out_dtype."""
    if stream is not None:
        return _on(stream, moe_linear, x, w, w_up, bias, bias_up, act, residual, out, out_dtype, z, z_up, ws,
                   use_workspace=use_workspace)
    (M, K), N = _matrix(x, "x"), _matrix(w, "w")[0]
    dev, bf, f32 = x.get_device(), torch.bfloat16, torch.float32
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    odt = out.dtype
    a = _choice(LINEAR_ACTS, act, "act")
    if ws is None and use_workspace:
        ws = alloc_linear_workspace(M, N, K, act, x.device)
    wsp, wsn = _ws(ws, dev)
    mn = (M, N)
    _launch((_lib or lib()).moe_linear, "moe_linear", dev, _take(x, "x", bf, (M, K), dev), _take(w, "w", bf, (N, K), dev),
            _take(w_up, "w_up", bf, (N, K), dev, True), _take(bias, "bias", f32, (N,), dev, True),
            _take(bias_up, "bias_up", f32, (N,), dev, True), _take(residual, "residual", odt, mn, dev, True), M, N, K, a,
            _choice(OUT_DTYPES, odt, "out's type"), _take(z, "z", bf, mn, dev, True), _take(z_up, "z_up", bf, mn, dev, True),
            _take(out, "out", odt, mn, dev), wsp, wsn)
    return out


def moe_linear_backward(d_out: torch.Tensor, x: torch.Tensor, w: torch.Tensor, w_up: Optional[torch.Tensor] = None,
                        act: str = "none", z: Optional[torch.Tensor] = None, z_up: Optional[torch.Tensor] = None,
                        d_x: Optional[torch.Tensor] = None, d_w: Optional[torch.Tensor] = None,
                        d_w_up: Optional[torch.Tensor] = None, d_bias: Optional[torch.Tensor] = None,
                        d_bias_up: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_linear, written into those of d_x, d_w, d_w_up, d_bias, d_bias_up that are given."""
    if stream is not None:
        return _on(stream, moe_linear_backward, d_out, x, w, w_up, act, z, z_up, d_x, d_w, d_w_up, d_bias, d_bias_up, ws)
    (M, K), N = _matrix(x, "x"), _matrix(w, "w")[0]
    dev, bf, f32 = x.get_device(), torch.bfloat16, torch.float32
    a = _choice(LINEAR_ACTS, act, "act")
    if ws is None:
        ws = alloc_linear_backward_workspace(M, N, K, act, x.device)
    wsp, wsn = _ws(ws, dev)
    mn, mk, nk = (M, N), (M, K), (N, K)
    _launch((_lib or lib()).moe_linear_backward, "moe_linear_backward", dev, _take(d_out, "d_out", d_out.dtype, mn, dev),
            _take(x, "x", bf, mk, dev), _take(w, "w", bf, nk, dev), _take(w_up, "w_up", bf, nk, dev, True),
            _take(z, "z", bf, mn, dev, True), _take(z_up, "z_up", bf, mn, dev, True), M, N, K, a,
            _choice(OUT_DTYPES, d_out.dtype, "d_out's type"), _take(d_x, "d_x", bf, mk, dev, True),
            _take(d_w, "d_w", bf, nk, dev, True), _take(d_w_up, "d_w_up", bf, nk, dev, True),
            _take(d_bias, "d_bias", f32, (N,), dev, True), _take(d_bias_up, "d_bias_up", f32, (N,), dev, True), wsp, wsn)
