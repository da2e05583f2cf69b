"""Python binding of libbra.so: argument marshalling only.

Every step of the forward pass runs in the library's CUDA kernels; these functions only
check tensor metadata, allocate outputs with torch and pass raw pointers and the current
CUDA stream through ctypes. If libbra.so is missing the first call raises: there is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
from typing import NamedTuple

import torch

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbra.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bra.h")

STATUS = {0: "BRA_OK", 1: "BRA_ERR_INVALID_ARG", 2: "BRA_ERR_UNSUPPORTED", 3: "BRA_ERR_CUDA",
          4: "BRA_ERR_INDEX", 5: "BRA_ERR_TIMEOUT"}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
NORM_KINDS = {"layer": 0, "rms": 1}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ATTEND_KERNELS = {"auto": 0, "simt": 1, "gather_mma": 2, "dense_mma": 3, "gather_umma": 4, "region_mma": 5}

_lib = None


class BraError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        name = STATUS.get(status, f"status {status}")
        super().__init__(f"{what}: {name}" + (f" ({detail})" if detail else ""))


def lib() -> ctypes.CDLL:
    """The loaded libbra.so (argument and result types set)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY):
        raise RuntimeError(f"{LIBRARY} is missing; build it with `python -m bi_level_routing_b200.build` "
                           "(there is no CPU fallback)")
    L = ctypes.CDLL(LIBRARY)
    vp, i32p, I = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_int
    L.bra_route.argtypes = [vp, vp, vp, I, I, I, I, I, I, I, vp]
    L.bra_attend.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_forward.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_forward_host.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_route_heads.argtypes = [vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_attend_heads.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_forward_heads.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_forward_auto_pad.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_lepe.argtypes = [vp, vp, vp, vp, I, I, I, I, I, vp]
    L.bra_forward_lepe.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_attend_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    F, I64 = ctypes.c_float, ctypes.c_int64
    L.bra_diff_attend.argtypes = [vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_forward_diff.argtypes = [vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_diff_attend_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp]
    L.bra_rope.argtypes = [vp, vp, vp, vp, vp, vp, I64, I64, I, I, I, I, I, I, I, I, I, F, I, vp]
    L.bra_norm_residual.argtypes = [vp, vp, vp, I, vp, vp, vp, vp, F, F, I, vp, vp, I, I, I, I, I, vp]
    L.bra_norm_residual_backward.argtypes = [vp, vp, vp, vp, vp, I, vp, vp, vp, vp, F, F, I, vp, vp, vp, vp, vp, vp, vp,
                                             I, I, I, I, I, vp]
    L.bra_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
    L.bra_set_attend_kernel.argtypes = [I]
    L.bra_set_max_ctas.argtypes = [I]
    L.bra_selected_attend_kernel.argtypes = [I, I, I, I, I, I, I, I]
    L.bra_check_device_error.argtypes = [vp]
    L.bra_route_scratch_bytes.argtypes = [I, I, I, I, I]
    L.bra_route_scratch_bytes.restype = ctypes.c_size_t
    L.bra_kernels_per_call.argtypes = [ctypes.c_char_p, I, I, I, I, I, I, I, I]
    L.bra_status_string.argtypes = [I]
    L.bra_status_string.restype = ctypes.c_char_p
    L.bra_last_error_message.restype = ctypes.c_char_p
    for name in ("bra_route", "bra_attend", "bra_forward", "bra_forward_host", "bra_set_attend_kernel", "bra_set_max_ctas",
                 "bra_route_heads", "bra_attend_heads", "bra_forward_heads", "bra_forward_auto_pad", "bra_lepe",
                 "bra_forward_lepe", "bra_attend_backward", "bra_selftest_wait_timeout", "bra_diff_attend",
                 "bra_forward_diff", "bra_diff_attend_backward", "bra_rope", "bra_norm_residual",
                 "bra_norm_residual_backward",
                 "bra_selected_attend_kernel", "bra_check_device_error", "bra_kernels_per_call"):
        getattr(L, name).restype = I
    _lib = L
    return L


def declared_symbols() -> list[str]:
    """Names of the functions include/bra.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(bra_\w+)\s*\(", text, flags=re.M)))


def _check(status: int, what: str):
    if status != 0:
        detail = lib().bra_last_error_message().decode() if status == 3 else ""
        raise BraError(status, what, detail)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _shape(x: torch.Tensor, name: str):
    if x.dim() != 4:
        raise ValueError(f"{name} must be [B, H, W, C], got shape {tuple(x.shape)}")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if x.dtype not in DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    return tuple(x.shape)


def _same(ref: torch.Tensor, *others):
    for name, t in others:
        if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
            raise ValueError(f"{name} must match q in shape, dtype and device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def route(q: torch.Tensor, k: torch.Tensor, n_win: int, topk: int, idx: torch.Tensor | None = None) -> torch.Tensor:
    """Routing index int32 [B, n_win^2, topk] (region means, affinity, top-k)."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k))
    R = n_win * n_win
    if idx is None:
        idx = torch.empty((B, R, topk), dtype=torch.int32, device=q.device)
    elif idx.shape != (B, R, topk) or idx.dtype != torch.int32 or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 [B, n_win^2, topk] tensor")
    _check(lib().bra_route(q.data_ptr(), k.data_ptr(), idx.data_ptr(), B, H, W, C, n_win, topk, DTYPES[q.dtype],
                           _stream(q.device)), "bra_route")
    return idx


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor, heads: int, n_win: int,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of every query over its region's routed keys; out has q's shape and dtype."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k), ("v", v))
    if idx.dim() != 3 or idx.dtype != torch.int32 or not idx.is_contiguous() or idx.device != q.device:
        raise ValueError("idx must be a contiguous int32 [B, n_win^2, topk] tensor on q's device")
    if out is None:
        out = torch.empty_like(q)
    _same(q, ("out", out))
    _check(lib().bra_attend(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(), B, H, W, C,
                            heads, n_win, idx.shape[-1], DTYPES[q.dtype], _stream(q.device)), "bra_attend")
    return out


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_win: int, topk: int, heads: int,
            out: torch.Tensor | None = None, idx: torch.Tensor | None = None):
    """The whole forward pass. Returns (out, idx)."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k), ("v", v))
    R = n_win * n_win
    if out is None:
        out = torch.empty_like(q)
    _same(q, ("out", out))
    if idx is None:
        idx = torch.empty((B, R, topk), dtype=torch.int32, device=q.device)
    elif idx.shape != (B, R, topk) or idx.dtype != torch.int32 or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 [B, n_win^2, topk] tensor")
    _check(lib().bra_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(), B, H, W, C,
                             heads, n_win, topk, DTYPES[q.dtype], _stream(q.device)), "bra_forward")
    return out, idx


def forward_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_win: int, topk: int, heads: int,
                 out: torch.Tensor | None = None, idx: torch.Tensor | None = None, device=None):
    """The forward pass on HOST tensors (pinned for full-speed copies): the library copies the
    inputs to the current CUDA device, runs the pass and copies out and idx back. Synchronous."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.is_cuda or not t.is_contiguous() or t.dim() != 4 or t.dtype not in DTYPES:
            raise ValueError(f"{name} must be a contiguous host [B, H, W, C] float32/bfloat16 tensor")
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must match")
    B, H, W, C = q.shape
    R = n_win * n_win
    if out is None:
        out = torch.empty_like(q, pin_memory=q.is_pinned())
    if idx is None:
        idx = torch.empty((B, R, topk), dtype=torch.int32, pin_memory=q.is_pinned())
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        _check(lib().bra_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(), B, H,
                                      W, C, heads, n_win, topk, DTYPES[q.dtype], _stream(device)), "bra_forward_host")
    return out, idx


def route_heads(q: torch.Tensor, k: torch.Tensor, n_win: int, topk: int, heads: int,
                idx: torch.Tensor | None = None) -> torch.Tensor:
    """Per-head routing index int32 [B, heads, n_win^2, min(topk, n_win^2)] (topk clamped to the
    number of regions, as the pages do)."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k))
    R = n_win * n_win
    topk = min(topk, R)
    if idx is None:
        idx = torch.empty((B, heads, R, topk), dtype=torch.int32, device=q.device)
    elif idx.shape != (B, heads, R, topk) or idx.dtype != torch.int32 or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 [B, heads, n_win^2, min(topk, n_win^2)] tensor")
    _check(lib().bra_route_heads(q.data_ptr(), k.data_ptr(), idx.data_ptr(), B, H, W, C, heads, n_win, topk,
                                 DTYPES[q.dtype], _stream(q.device)), "bra_route_heads")
    return idx


def attend_heads(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor, n_win: int,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention where head h gathers the regions of its own rows idx [B, heads, R, topk]."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k), ("v", v))
    if idx.dim() != 4 or idx.dtype != torch.int32 or not idx.is_contiguous() or idx.device != q.device:
        raise ValueError("idx must be a contiguous int32 [B, heads, n_win^2, topk] tensor on q's device")
    if out is None:
        out = torch.empty_like(q)
    _same(q, ("out", out))
    _check(lib().bra_attend_heads(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(), B, H, W,
                                  C, idx.shape[1], n_win, idx.shape[-1], DTYPES[q.dtype], _stream(q.device)),
           "bra_attend_heads")
    return out


def forward_heads(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_win: int, topk: int, heads: int,
                  out: torch.Tensor | None = None, idx: torch.Tensor | None = None):
    """The forward pass with per-head routing. Returns (out, idx [B, heads, R, min(topk, R)])."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k), ("v", v))
    R = n_win * n_win
    topk = min(topk, R)
    if out is None:
        out = torch.empty_like(q)
    _same(q, ("out", out))
    if idx is None:
        idx = torch.empty((B, heads, R, topk), dtype=torch.int32, device=q.device)
    _check(lib().bra_forward_heads(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(), B, H,
                                   W, C, heads, n_win, topk, DTYPES[q.dtype], _stream(q.device)), "bra_forward_heads")
    return out, idx


def forward_auto_pad(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_win: int, topk: int, heads: int,
                     out: torch.Tensor | None = None, idx: torch.Tensor | None = None):
    """The forward pass on any H x W: the map is taken as zero-padded at the bottom and right to
    multiples of n_win (nothing is copied), and out has q's shape. Returns (out, idx)."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k), ("v", v))
    R = n_win * n_win
    if out is None:
        out = torch.empty_like(q)
    _same(q, ("out", out))
    if idx is None:
        idx = torch.empty((B, R, topk), dtype=torch.int32, device=q.device)
    _check(lib().bra_forward_auto_pad(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(), B, H,
                                      W, C, heads, n_win, topk, DTYPES[q.dtype], _stream(q.device)),
           "bra_forward_auto_pad")
    return out, idx


def lepe(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """x + 5x5 depthwise convolution of x (zero padding 2) + bias; weight fp32 [C, 5, 5], bias fp32 [C]."""
    B, H, W, C = _shape(x, "x")
    for name, t, shape in (("weight", weight, (C, 5, 5)), ("bias", bias, (C,))):
        if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous() or t.device != x.device:
            raise ValueError(f"{name} must be a contiguous float32 {shape} tensor on x's device")
    if out is None:
        out = torch.empty_like(x)
    _same(x, ("out", out))
    _check(lib().bra_lepe(x.data_ptr(), weight.data_ptr(), bias.data_ptr(), out.data_ptr(), B, H, W, C,
                          DTYPES[x.dtype], _stream(x.device)), "bra_lepe")
    return out


def forward_lepe(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_win: int, topk: int, heads: int,
                 weight: torch.Tensor, bias: torch.Tensor, attn: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, idx: torch.Tensor | None = None):
    """The forward pass followed by the LePE epilogue. Returns (out, attn, idx): attn is the
    attention output, out = attn + lepe(attn)."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k), ("v", v))
    R = n_win * n_win
    attn = torch.empty_like(q) if attn is None else attn
    out = torch.empty_like(q) if out is None else out
    _same(q, ("attn", attn), ("out", out))
    if idx is None:
        idx = torch.empty((B, R, topk), dtype=torch.int32, device=q.device)
    _check(lib().bra_forward_lepe(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), attn.data_ptr(),
                                  out.data_ptr(), weight.data_ptr(), bias.data_ptr(), B, H, W, C, heads, n_win, topk,
                                  DTYPES[q.dtype], _stream(q.device)), "bra_forward_lepe")
    return out, attn, idx


def attend_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor, dout: torch.Tensor,
                    heads: int, n_win: int, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                    dv: torch.Tensor | None = None):
    """(dq, dk, dv), float32 [B, H, W, C]: gradients of sum(dout * attend(q, k, v, idx)), idx fixed."""
    B, H, W, C = _shape(q, "q")
    _same(q, ("k", k), ("v", v), ("dout", dout))
    if idx.dim() != 3 or idx.dtype != torch.int32 or not idx.is_contiguous() or idx.device != q.device:
        raise ValueError("idx must be a contiguous int32 [B, n_win^2, topk] tensor on q's device")
    grads = []
    for name, g in (("dq", dq), ("dk", dk), ("dv", dv)):
        if g is None:
            g = torch.empty((B, H, W, C), dtype=torch.float32, device=q.device)
        elif g.shape != (B, H, W, C) or g.dtype != torch.float32 or not g.is_contiguous() or g.device != q.device:
            raise ValueError(f"{name} must be a contiguous float32 [B, H, W, C] tensor on q's device")
        grads.append(g)
    dq, dk, dv = grads
    _check(lib().bra_attend_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), dout.data_ptr(),
                                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, W, C, heads, n_win,
                                     idx.shape[-1], DTYPES[q.dtype], _stream(q.device)), "bra_attend_backward")
    return dq, dk, dv


def _on_device(t: torch.Tensor, fn, *args) -> int:
    """fn(*args, stream) with t's device current, on its current stream: the tensors' device need not be the
    caller's current one."""
    index = t.get_device()
    if torch.cuda.current_device() == index:
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))


def _alike(ref: torch.Tensor, what: str, *others):
    """The checks of _same, for the (name, tensor) pairs whose tensor is not None."""
    shape, dtype, device = ref.shape, ref.dtype, ref.get_device()
    for name, t in others:
        if t is None:
            continue
        if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
            raise ValueError(f"{name} must match {what} in shape, dtype and device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _routed(idx: torch.Tensor, q: torch.Tensor, n_win: int) -> int:
    """Checks a routing index for q and returns its topk."""
    shape = idx.shape
    if (len(shape) != 3 or shape[0] != q.shape[0] or shape[1] != n_win * n_win or idx.dtype is not torch.int32
            or not idx.is_contiguous() or idx.get_device() != q.get_device()):
        raise ValueError("idx must be a contiguous int32 [B, n_win^2, topk] tensor on q's device")
    return shape[2]


def _vector(t: torch.Tensor | None, name: str, device: int, *shapes):
    """The address of a contiguous fp32 tensor of one of `shapes` on `device`, or None for None."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape not in shapes or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {' or '.join(map(str, shapes))} on "
                         "the maps' device")
    return t.data_ptr()


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def diff_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor, lam: torch.Tensor, heads: int,
                n_win: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Differential attention over the routed regions: per head the map of the first half of its q and k
    channels minus lam[head] times the map of the second half, times v. lam: float32 [heads]."""
    B, H, W, C = _shape(q, "q")
    _alike(q, "q", ("k", k), ("v", v), ("out", out))
    topk = _routed(idx, q, n_win)
    weight = _vector(lam, "lam", q.get_device(), (heads,))
    if out is None:
        out = torch.empty_like(q)
    _check(_on_device(q, lib().bra_diff_attend, q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), weight,
                      out.data_ptr(), B, H, W, C, heads, n_win, topk, DTYPES[q.dtype]), "bra_diff_attend")
    return out


def forward_diff(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, n_win: int, topk: int, heads: int,
                 out: torch.Tensor | None = None, idx: torch.Tensor | None = None):
    """Routing, then differential attention. Returns (out, idx)."""
    B, H, W, C = _shape(q, "q")
    _alike(q, "q", ("k", k), ("v", v), ("out", out))
    weight = _vector(lam, "lam", q.get_device(), (heads,))
    if out is None:
        out = torch.empty_like(q)
    if idx is None:
        idx = torch.empty((B, n_win * n_win, topk), dtype=torch.int32, device=q.device)
    if _routed(idx, q, n_win) != topk:
        raise ValueError("idx must be a contiguous int32 [B, n_win^2, topk] tensor")
    _check(_on_device(q, lib().bra_forward_diff, q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), weight,
                      out.data_ptr(), B, H, W, C, heads, n_win, topk, DTYPES[q.dtype]), "bra_forward_diff")
    return out, idx


def diff_attend_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor, lam: torch.Tensor,
                         dout: torch.Tensor, heads: int, n_win: int, dq: torch.Tensor | None = None,
                         dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                         dlam: torch.Tensor | None = None):
    """(dq, dk, dv, dlam): gradients of sum(dout * diff_attend(q, k, v, idx, lam)), idx fixed. dq, dk and dv
    have q's type, dlam is float32 [heads]; the same bits on every run."""
    B, H, W, C = _shape(q, "q")
    _alike(q, "q", ("k", k), ("v", v), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv))
    topk = _routed(idx, q, n_win)
    weight = _vector(lam, "lam", q.get_device(), (heads,))
    dq, dk, dv = (torch.empty_like(q) if t is None else t for t in (dq, dk, dv))
    if dlam is None:
        dlam = torch.empty_like(lam)
    _check(_on_device(q, lib().bra_diff_attend_backward, q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), weight,
                      dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                      _vector(dlam, "dlam", q.get_device(), (heads,)), B, H, W, C, heads, n_win, topk, DTYPES[q.dtype]),
           "bra_diff_attend_backward")
    return dq, dk, dv, dlam


def rope(q: torch.Tensor, k: torch.Tensor | None, freqs: torch.Tensor, heads: int, layout: str = "half", axes: int = 2,
         origin: tuple[int, int] = (0, 0), pos: torch.Tensor | None = None, mscale: float = 1.0, inverse: bool = False,
         q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
    """Rotary positions of q and k (k may be None). The first 2 * axes * len(freqs) channels of each head are
    turned: pairs (i, i + n) of each axis' block ("half") or (2i, 2i + 1) ("interleaved") by position * freqs[i].
    Positions: the token's row and column (axes=2) or raster number (axes=1) from `origin`, or pos, int32
    [B, H, W, axes]. inverse=True takes gradients back. q_out may be q, k_out k (in place).
    Returns (q_out, k_out). See rope_frequencies for freqs and mscale."""
    B, H, W, C = _shape(q, "q")
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    _alike(q, "q", ("k", k), ("q_out", q_out), ("k_out", k_out))
    n = freqs.numel()
    table = _vector(freqs, "freqs", q.get_device(), (n,))
    if pos is not None and (pos.shape != (B, H, W, axes) or pos.dtype is not torch.int32 or not pos.is_contiguous()
                            or pos.get_device() != q.get_device()):
        raise ValueError("pos must be a contiguous int32 [B, H, W, axes] tensor on q's device")
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    if q_out is None:
        q_out = torch.empty_like(q)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k)
    _check(_on_device(q, lib().bra_rope, q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out), table, _ptr(pos),
                      int(origin[0]), int(origin[1]), B, H, W, C, heads, n, axes, ROPE_LAYOUTS[layout], int(inverse),
                      float(mscale), DTYPES[q.dtype]), "bra_rope")
    return q_out, k_out


def rope_frequencies(n: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained_extent: int | None = None, device=None) -> tuple[torch.Tensor, float]:
    """(freqs float32 [n], mscale) for `rope`: freqs[i] = base^(-i / n), stretched by `factor` for maps or
    sequences that much longer than the trained ones:
      "linear"  every frequency divided by factor (positions interpolated);
      "ntk"     base multiplied by factor^(n / (n - 1)): the fastest stays, the slowest is divided by factor;
      "yarn"    frequencies that turn more than 32 times over trained_extent positions stay, those that turn
                less than once are divided by factor, a linear ramp (in the number of the pair) between, from
                pair 0 where none turns 32 times; mscale = 0.1 ln(factor) + 1."""
    if n <= 0 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("n must be positive, base above 1 and factor at least 1")
    i = torch.arange(n, dtype=torch.float64)
    mscale = 1.0
    if scaling == "ntk" and n > 1:
        base = base * factor ** (n / (n - 1))
    freqs = base ** (-i / n)
    if scaling == "linear" or (scaling == "ntk" and n == 1):
        freqs = freqs / factor
    elif scaling == "yarn":
        if not trained_extent or trained_extent <= 0:
            raise ValueError("yarn scaling needs trained_extent, the positions seen in training")
        # the (real) pair numbers that turn 32 times and once over the trained extent
        fast, slow = (n * math.log(trained_extent / (turns * 2 * math.pi)) / math.log(base) for turns in (32, 1))
        low, high = max(math.floor(fast), 0), math.ceil(slow)  # high may lie past the table: then no pair turns less than once
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        ramp[i > slow] = 1.0  # also where not even pair 0 turns once
        freqs = freqs * (1 - ramp) + freqs / factor * ramp
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling must be none, linear, ntk or yarn, got {scaling!r}")
    return freqs.float().to(device), mscale


def _norm_arguments(x, h, gate, post_weight, post_bias, pre_weight, pre_bias, alpha, eps, kind):
    """Checks the arguments both norm calls share; returns (shape, those from the gate to the kind for the C call)."""
    B, H, W, C = _shape(x, "x")
    if kind not in NORM_KINDS:
        raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}, got {kind!r}")
    device, per_channel = x.get_device(), (C,)
    gates = 0 if gate is None else 1 if gate.dim() == 1 else B
    return (B, H, W, C), (_vector(gate, "gate", device, per_channel, (B, C)), gates,
                          _vector(post_weight, "post_weight", device, per_channel),
                          _vector(post_bias, "post_bias", device, per_channel),
                          _vector(pre_weight, "pre_weight", device, per_channel),
                          _vector(pre_bias, "pre_bias", device, per_channel), float(alpha), float(eps), NORM_KINDS[kind])


def norm_residual(x: torch.Tensor, h: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
                  pre_weight: torch.Tensor | None = None, pre_bias: torch.Tensor | None = None, alpha: float = 1.0,
                  eps: float = 1e-6, kind: str = "layer", s_out: torch.Tensor | None = None,
                  y_out: torch.Tensor | None = None):
    """The norms around a block in one pass: s = alpha * x + gate * (norm(h) * post_weight + post_bias) and
    y = norm(s) * pre_weight + pre_bias, norm a LayerNorm or an RMS norm (kind "layer", "rms"). Without
    post_weight h is taken as it is, without h s = alpha * x, without pre_weight there is no y. Weights, biases:
    float32 [C]; gate: float32 [C] or, one for each image, [B, C]. Returns (s, y); s is None where h is None
    (unless s_out is given), y where pre_weight is None."""
    shape, middle = _norm_arguments(x, h, gate, post_weight, post_bias, pre_weight, pre_bias, alpha, eps, kind)
    _alike(x, "x", ("h", h), ("s_out", s_out), ("y_out", y_out))
    if h is not None and s_out is None:
        s_out = torch.empty_like(x)
    if pre_weight is not None and y_out is None:
        y_out = torch.empty_like(x)
    elif pre_weight is None and y_out is not None:
        raise ValueError("y_out without pre_weight")
    _check(_on_device(x, lib().bra_norm_residual, x.data_ptr(), _ptr(h), *middle, _ptr(s_out), _ptr(y_out), *shape,
                      DTYPES[x.dtype]), "bra_norm_residual")
    return s_out, y_out


class NormGrads(NamedTuple):
    """Gradients of norm_residual by its inputs, None for inputs that were not given."""
    dx: torch.Tensor
    dh: torch.Tensor | None
    dgate: torch.Tensor | None
    dpost_weight: torch.Tensor | None
    dpost_bias: torch.Tensor | None
    dpre_weight: torch.Tensor | None
    dpre_bias: torch.Tensor | None


def norm_residual_backward(x: torch.Tensor, h: torch.Tensor | None, dy: torch.Tensor | None, ds: torch.Tensor | None,
                           gate: torch.Tensor | None = None, post_weight: torch.Tensor | None = None,
                           post_bias: torch.Tensor | None = None, pre_weight: torch.Tensor | None = None,
                           pre_bias: torch.Tensor | None = None, alpha: float = 1.0, eps: float = 1e-6,
                           kind: str = "layer", dx: torch.Tensor | None = None,
                           dh: torch.Tensor | None = None) -> NormGrads:
    """Gradients of sum(ds * s) + sum(dy * y) of norm_residual with the same arguments. dy is given exactly where
    pre_weight is; ds may be None (no gradient of s). dx and dh have x's type, the others are float32 of their
    inputs' shapes; the same bits on every run."""
    shape, middle = _norm_arguments(x, h, gate, post_weight, post_bias, pre_weight, pre_bias, alpha, eps, kind)
    _alike(x, "x", ("h", h), ("dy", dy), ("ds", ds), ("dx", dx), ("dh", dh))
    if dx is None:
        dx = torch.empty_like(x)
    if h is not None and dh is None:
        dh = torch.empty_like(x)
    elif h is None and dh is not None:
        raise ValueError("dh without h")
    dgate, dpw, dpb, dnw, dnb = (None if t is None else torch.empty_like(t)
                                 for t in (gate, post_weight, post_bias, pre_weight, pre_bias))
    _check(_on_device(x, lib().bra_norm_residual_backward, x.data_ptr(), _ptr(h), _ptr(dy), _ptr(ds), *middle,
                      dx.data_ptr(), _ptr(dh), _ptr(dgate), _ptr(dpw), _ptr(dpb), _ptr(dnw), _ptr(dnb), *shape,
                      DTYPES[x.dtype]), "bra_norm_residual_backward")
    return NormGrads(dx, dh, dgate, dpw, dpb, dnw, dnb)


def check_device_error(device=None) -> int:
    """Synchronises the current stream and returns (and clears) the device error status."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        return lib().bra_check_device_error(_stream(device))


def set_attend_kernel(name: str):
    """Force one attention kernel ("simt", "gather_mma", "dense_mma", "gather_umma") or release ("auto")."""
    _check(lib().bra_set_attend_kernel(ATTEND_KERNELS[name]), "bra_set_attend_kernel")


def set_max_ctas(n: int):
    """Cap the persistent attention kernels' grid at n CTAs (0 = no cap); the result does not change."""
    _check(lib().bra_set_max_ctas(int(n)), "bra_set_max_ctas")


def selected_attend_kernel(B, H, W, C, heads, n_win, topk, dtype) -> str | None:
    code = lib().bra_selected_attend_kernel(B, H, W, C, heads, n_win, topk, DTYPES[dtype])
    return {v: k for k, v in ATTEND_KERNELS.items()}.get(code)


def kernels_per_call(entry_point: str, B, H, W, C, heads, n_win, topk, dtype) -> int:
    return lib().bra_kernels_per_call(entry_point.encode(), B, H, W, C, heads, n_win, topk, DTYPES[dtype])


def route_scratch_bytes(B, H, W, C, n_win) -> int:
    return int(lib().bra_route_scratch_bytes(B, H, W, C, n_win))
