"""nvfp4_sm_skinny_gb300: small-M skinny GEMM with a deterministic split-K
reduction and its fused epilogues (pre-expert RMSNorm + NVFP4, attention
boundary dual norm) for GB300 (sm_103a).

This module is a thin ctypes binding over ``libsk.so`` (C ABI in
``include/sk.h``). It only marshals torch tensors (device pointers, the current
stream) into the C calls and allocates outputs the caller did not pass; every
step of the computation runs in the library's CUDA kernels. There is no CPU or
PyTorch fallback: if ``libsk.so`` is missing or cannot be loaded, the first
call raises.

Build the library with ``python -c "import __graft_entry__ as g; g.build()"``
or ``python nvfp4_sm_skinny_gb300/build.py``.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsk.so")

SK_OK = 0
SK_ERR_INVALID_ARG = 1
SK_ERR_UNSUPPORTED = 2
SK_ERR_ARCH = 3
SK_ERR_WORKSPACE = 4
SK_ERR_CUDA = 5
SK_ERR_DEVICE_TIMEOUT = 6
MAX_M = 16

_lock = threading.Lock()
_lib = None


class SkError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[sk status {status}] {message}")
        self.status = status


class SkValueError(ValueError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[sk status {status}] {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libsk.so (raises if it was not built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libsk.so not found at {LIB_PATH}: build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        i64 = ctypes.c_int64
        sig = {
            "sk_last_error": ([], ctypes.c_char_p),
            "sk_version": ([], i),
            "sk_gemm_splits": ([i, i, i, i], i),
            "sk_gemm_supported": ([i, i, i, i], i),
            "sk_gemm_bf16": ([vp, vp, vp, i, i, i, i, vp], i),
            "sk_gemm_prefetch_next": ([vp, i, i], i),
            "sk_gemm_bf16_ex": ([vp, vp, vp, i, i, i, i, ctypes.c_uint, vp], i),
            "sk_rmsnorm_nvfp4": ([vp, vp, f, f, vp, vp, vp, vp, i, i, vp], i),
            "sk_gemm_rmsnorm_nvfp4_workspace": ([i, i], sz),
            "sk_gemm_rmsnorm_nvfp4": ([vp, vp, vp, f, f, vp, vp, vp, vp, vp, sz, i, i, i, i, vp], i),
            "sk_nvfp4_quantize": ([vp, vp, vp, vp, i, i, vp], i),
            "sk_rmsnorm_bf16": ([vp, vp, f, f, vp, i, i, vp], i),
            "sk_gemm_rmsnorm_bf16": ([vp, vp, vp, f, f, vp, vp, sz, i, i, i, i, vp], i),
            "sk_dual_norm_residual": ([vp, vp, vp, f, vp, vp, vp, f, f, f, f, i, i, vp], i),
            "sk_gemm_dual_norm_workspace": ([i, i], sz),
            "sk_gemm_dual_norm": ([vp, vp, vp, vp, f, vp, vp, vp, f, f, f, f, vp, sz, i, i, i, i, vp], i),
            "sk_gemm_rmsnorm_nvfp4_static": ([vp, vp, vp, f, f, vp, vp, vp, vp, i, i, i, i, vp], i),
            "sk_gemm_nvfp4w_bf16": ([vp, vp, vp, vp, vp, i, i, i, i, vp], i),
            "sk_gemm_nvfp4w_supported": ([i, i, i, i], i),
            "sk_gemm_nvfp4w_splits": ([i, i, i, i], i),
            "sk_route": ([vp, i, vp, vp, vp, i, i, i, i, i, i, i, f, vp], i),
            "sk_int8_quantize": ([vp, vp, vp, i, i, vp], i),
            "sk_gemm_int8": ([vp, vp, vp, vp, vp, i, i, i, i, vp], i),
            "sk_gemm_int8_supported": ([i, i, i, i], i),
            "sk_experts_int8_workspace": ([i, i, i, i], sz),
            "sk_experts_int8": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, vp], i),
            "sk_kv_block_bytes": ([i, i], sz),
            "sk_kv_append": ([vp] * 7 + [i] * 7 + [i64, i64, vp], i),
            "sk_kv_append_ex": ([vp] * 9 + [i] * 7 + [i64, i64, vp], i),
            "sk_attn_nvfp4_workspace": ([i] * 5, sz),
            "sk_attn_nvfp4": ([vp] * 9 + [sz] + [i] * 8 + [i64, f, i, vp], i),
            "sk_kv_resize_workspace": ([i, i], sz),
            "sk_kv_resize": ([vp] * 7 + [sz] + [i] * 7 + [vp], i),
            "sk_kv_fork": ([vp] * 5 + [i] * 4 + [vp], i),
            "sk_kv_compact_workspace": ([i], sz),
            "sk_kv_compact": ([vp] * 6 + [sz] + [i] * 7 + [vp], i),
            "sk_device_status": ([ctypes.POINTER(ctypes.c_uint32), i], i),
            "sk_convert_probe": ([i, vp, vp, i, vp], i),
            "sk_wait_probe": ([ctypes.c_uint, vp], i),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return L


def last_error() -> str:
    return lib().sk_last_error().decode()


def _check(status: int) -> None:
    if status == SK_OK:
        return
    msg = last_error()
    if status in (SK_ERR_INVALID_ARG, SK_ERR_UNSUPPORTED, SK_ERR_WORKSPACE):
        raise SkValueError(status, msg)
    raise SkError(status, msg)


def _ptr(t) -> ctypes.c_void_p | None:
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, shape, name):
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, needs {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, needs {tuple(shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: needs a contiguous CUDA tensor")


def version() -> int:
    return int(lib().sk_version())


def gemm_supported(m: int, n: int, k: int, splits: int = 0) -> str | None:
    """None if (m, n, k, splits) has a launch, else the reason."""
    st = lib().sk_gemm_supported(m, n, k, splits)
    return None if st == SK_OK else last_error()


def gemm_splits(m: int, n: int, k: int, splits: int = 0) -> int:
    s = int(lib().sk_gemm_splits(m, n, k, splits))
    if s == 0:
        raise SkValueError(SK_ERR_UNSUPPORTED, last_error())
    return s


# ----------------------------------------------------------------- GEMM ----
GEMM_X_READY = 0x1


def gemm_bf16(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
              splits: int = 0, stream=None, x_ready: bool = False) -> torch.Tensor:
    """out[m, n] = x[m, k] @ w[n, k]^T (BF16 in/out, FP32 accumulate).
    ``x_ready``: no kernel that writes x can still be running when this GEMM
    starts (x written by host copies, or by kernels before a copy, event wait,
    non-overlapped launch or synchronisation), so the GEMM reads it without
    waiting for the kernel ahead of it (sk_gemm_bf16_ex, SK_GEMM_X_READY)."""
    m, k = x.shape
    n = w.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(w, torch.bfloat16, (n, k), "w")
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (m, n), "out")
    if x_ready:
        _check(lib().sk_gemm_bf16_ex(_ptr(x), _ptr(w), _ptr(out), m, n, k, splits, GEMM_X_READY,
                                     _stream(stream)))
    else:
        _check(lib().sk_gemm_bf16(_ptr(x), _ptr(w), _ptr(out), m, n, k, splits, _stream(stream)))
    return out


def gemm_prefetch_next(w_next: torch.Tensor | None) -> None:
    """Hint for the next GEMM this thread enqueues: once it has issued its own
    weight copies, it starts the first weight stages of the GEMM with weight
    ``w_next`` [n, k] (BF16) towards L2. ``None`` clears the hint."""
    if w_next is None:
        _check(lib().sk_gemm_prefetch_next(None, 0, 0))
        return
    _need(w_next, torch.bfloat16, tuple(w_next.shape), "w_next")
    n, k = w_next.shape
    _check(lib().sk_gemm_prefetch_next(_ptr(w_next), n, k))


# -------------------------------------------------------- RMSNorm + NVFP4 ----
def _nvfp4_outputs(m, n, device, a, a_sf):
    if a is None:
        a = torch.empty(m, n // 2, dtype=torch.uint8, device=device)
    if a_sf is None:
        a_sf = torch.empty(m, n // 16, dtype=torch.uint8, device=device)
    _need(a, torch.uint8, (m, n // 2), "a")
    _need(a_sf, torch.uint8, (m, n // 16), "a_sf")
    return a, a_sf


def rmsnorm_nvfp4(y, norm_w, eps: float, gain_center: float, global_scale, a=None, a_sf=None,
                  z_out=None, stream=None):
    """(a, a_sf, z_out): pre-expert RMSNorm of BF16 y [m, n] then NVFP4.
    ``z_out`` may be a tensor, True (allocate) or None (not stored)."""
    m, n = y.shape
    _need(y, torch.bfloat16, (m, n), "y")
    _need(norm_w, torch.bfloat16, (n,), "norm_w")
    _need(global_scale, torch.float32, (1,), "global_scale")
    a, a_sf = _nvfp4_outputs(m, n, y.device, a, a_sf)
    if z_out is True:
        z_out = torch.empty(m, n, dtype=torch.bfloat16, device=y.device)
    if z_out is not None:
        _need(z_out, torch.bfloat16, (m, n), "z_out")
    _check(lib().sk_rmsnorm_nvfp4(_ptr(y), _ptr(norm_w), eps, gain_center, _ptr(global_scale),
                                  _ptr(a), _ptr(a_sf), _ptr(z_out), m, n, _stream(stream)))
    return a, a_sf, z_out


def rmsnorm_bf16(y, norm_w, eps: float, gain_center: float, out=None, stream=None):
    """z BF16 [m, n]: pre-expert RMSNorm of a BF16 edge layer (no NVFP4)."""
    m, n = y.shape
    _need(y, torch.bfloat16, (m, n), "y")
    _need(norm_w, torch.bfloat16, (n,), "norm_w")
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=y.device)
    _need(out, torch.bfloat16, (m, n), "out")
    _check(lib().sk_rmsnorm_bf16(_ptr(y), _ptr(norm_w), eps, gain_center, _ptr(out), m, n,
                                 _stream(stream)))
    return out


def gemm_rmsnorm_bf16(x, w, norm_w, eps: float, gain_center: float, out=None, workspace=None,
                      splits: int = 0, stream=None):
    """(z, workspace): the pooler GEMM then the pre-expert RMSNorm of a BF16
    edge layer. The workspace (uint8) holds the BF16 GEMM output on return."""
    m, k = x.shape
    n = w.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(w, torch.bfloat16, (n, k), "w")
    _need(norm_w, torch.bfloat16, (n,), "norm_w")
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (m, n), "out")
    if workspace is None:
        workspace = torch.empty(gemm_rmsnorm_nvfp4_workspace(m, n), dtype=torch.uint8,
                                device=x.device)
    _check(lib().sk_gemm_rmsnorm_bf16(
        _ptr(x), _ptr(w), _ptr(norm_w), eps, gain_center, _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), m, n, k, splits, _stream(stream)))
    return out, workspace


def gemm_rmsnorm_nvfp4_workspace(m: int, n: int) -> int:
    return int(lib().sk_gemm_rmsnorm_nvfp4_workspace(m, n))


def gemm_rmsnorm_nvfp4(x, w, norm_w, eps: float, gain_center: float, global_scale, a=None,
                       a_sf=None, z_out=None, workspace=None, splits: int = 0, stream=None):
    """(a, a_sf, z_out, workspace): the pooler GEMM, pre-expert RMSNorm and
    NVFP4. The workspace (uint8) holds the BF16 GEMM output on return."""
    m, k = x.shape
    n = w.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(w, torch.bfloat16, (n, k), "w")
    _need(norm_w, torch.bfloat16, (n,), "norm_w")
    _need(global_scale, torch.float32, (1,), "global_scale")
    a, a_sf = _nvfp4_outputs(m, n, x.device, a, a_sf)
    if z_out is True:
        z_out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    if z_out is not None:
        _need(z_out, torch.bfloat16, (m, n), "z_out")
    need = gemm_rmsnorm_nvfp4_workspace(m, n)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check(lib().sk_gemm_rmsnorm_nvfp4(
        _ptr(x), _ptr(w), _ptr(norm_w), eps, gain_center, _ptr(global_scale), _ptr(a), _ptr(a_sf),
        _ptr(z_out), _ptr(workspace), workspace.numel() * workspace.element_size(), m, n, k,
        splits, _stream(stream)))
    return a, a_sf, z_out, workspace


STATIC_SCRATCH_BYTES = 16 * 8192 * 2


def gemm_rmsnorm_nvfp4_static(x, w, norm_w, eps: float, gain_center: float, global_scale, a,
                              a_sf, z_out=None, splits: int = 0, stream=None):
    """The pooler call without a workspace (the library's static device
    scratch holds the GEMM output; m * n <= 131072). The caller passes every
    output; nothing is allocated."""
    m, k = x.shape
    n = w.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(w, torch.bfloat16, (n, k), "w")
    _need(norm_w, torch.bfloat16, (n,), "norm_w")
    _need(global_scale, torch.float32, (1,), "global_scale")
    _need(a, torch.uint8, (m, n // 2), "a")
    _need(a_sf, torch.uint8, (m, n // 16), "a_sf")
    if z_out is not None:
        _need(z_out, torch.bfloat16, (m, n), "z_out")
    _check(lib().sk_gemm_rmsnorm_nvfp4_static(
        _ptr(x), _ptr(w), _ptr(norm_w), eps, gain_center, _ptr(global_scale), _ptr(a), _ptr(a_sf),
        _ptr(z_out), m, n, k, splits, _stream(stream)))
    return a, a_sf, z_out


def nvfp4_quantize(z, global_scale, a=None, a_sf=None, stream=None):
    """(a, a_sf): NVFP4 of BF16 z [m, n]."""
    m, n = z.shape
    _need(z, torch.bfloat16, (m, n), "z")
    _need(global_scale, torch.float32, (1,), "global_scale")
    a, a_sf = _nvfp4_outputs(m, n, z.device, a, a_sf)
    _check(lib().sk_nvfp4_quantize(_ptr(z), _ptr(global_scale), _ptr(a), _ptr(a_sf), m, n,
                                   _stream(stream)))
    return a, a_sf


# ------------------------------------------------------------- dual norm ----
def dual_norm_residual(partial, resid, post_w, alpha: float, beta, pre_w, out=None,
                       eps_post: float = 1e-6, eps_pre: float = 1e-6, gc_post: float = 0.0,
                       gc_pre: float = 0.0, stream=None):
    """out: post_attn_norm(partial), gated add into resid (FP32, in place),
    pre_ffn_norm into BF16 out."""
    m, h = partial.shape
    _need(partial, torch.bfloat16, (m, h), "partial")
    _need(resid, torch.float32, (m, h), "resid")
    if post_w is not None:
        _need(post_w, torch.bfloat16, (h,), "post_w")
    _need(beta, torch.bfloat16, (h,), "beta")
    _need(pre_w, torch.bfloat16, (h,), "pre_w")
    if out is None:
        out = torch.empty(m, h, dtype=torch.bfloat16, device=partial.device)
    _need(out, torch.bfloat16, (m, h), "out")
    _check(lib().sk_dual_norm_residual(_ptr(partial), _ptr(resid), _ptr(post_w), alpha, _ptr(beta),
                                       _ptr(pre_w), _ptr(out), eps_post, eps_pre, gc_post, gc_pre,
                                       m, h, _stream(stream)))
    return out


def gemm_dual_norm_workspace(m: int, n: int) -> int:
    return int(lib().sk_gemm_dual_norm_workspace(m, n))


def gemm_dual_norm(x, w, resid, post_w, alpha: float, beta, pre_w, out=None,
                   eps_post: float = 1e-6, eps_pre: float = 1e-6, gc_post: float = 0.0,
                   gc_pre: float = 0.0, workspace=None, splits: int = 0, stream=None):
    """(out, workspace): o_proj GEMM then the dual norm. The workspace holds the
    BF16 partial on return."""
    m, k = x.shape
    n = w.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(w, torch.bfloat16, (n, k), "w")
    _need(resid, torch.float32, (m, n), "resid")
    if post_w is not None:
        _need(post_w, torch.bfloat16, (n,), "post_w")
    _need(beta, torch.bfloat16, (n,), "beta")
    _need(pre_w, torch.bfloat16, (n,), "pre_w")
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (m, n), "out")
    need = gemm_dual_norm_workspace(m, n)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check(lib().sk_gemm_dual_norm(
        _ptr(x), _ptr(w), _ptr(resid), _ptr(post_w), alpha, _ptr(beta), _ptr(pre_w), _ptr(out),
        eps_post, eps_pre, gc_post, gc_pre, _ptr(workspace),
        workspace.numel() * workspace.element_size(), m, n, k, splits, _stream(stream)))
    return out, workspace


# ------------------------------------------------- weight-only NVFP4 GEMM ----
def gemm_nvfp4w_supported(m: int, n: int, k: int, splits: int = 0) -> str | None:
    """None if the weight-only NVFP4 GEMM has a launch for the shape, else why."""
    st = lib().sk_gemm_nvfp4w_supported(m, n, k, splits)
    return None if st == SK_OK else last_error()


def gemm_nvfp4w_splits(m: int, n: int, k: int, splits: int = 0) -> int:
    s = int(lib().sk_gemm_nvfp4w_splits(m, n, k, splits))
    if s == 0:
        raise SkValueError(SK_ERR_UNSUPPORTED, last_error())
    return s


def gemm_nvfp4w(x, wq, wsf, w_scale, out=None, splits: int = 0, stream=None):
    """out[m, n] = bf16(w_scale * x[m, k] @ W^T), W[n, k] = e2m1(wq) * e4m3(wsf):
    wq uint8 [n, k/2] (column 2c in the low nibble), wsf uint8 [n, k/16]
    (float8_e4m3fn bits), w_scale float32 [1] on the device."""
    m, k = x.shape
    n = wq.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(wq, torch.uint8, (n, k // 2), "wq")
    _need(wsf, torch.uint8, (n, k // 16), "wsf")
    _need(w_scale, torch.float32, (1,), "w_scale")
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (m, n), "out")
    _check(lib().sk_gemm_nvfp4w_bf16(_ptr(x), _ptr(wq), _ptr(wsf), _ptr(w_scale), _ptr(out), m, n,
                                     k, splits, _stream(stream)))
    return out


# ------------------------------------------------ int8 and routed experts ----
SCORES = {"softmax": 0, "sigmoid": 1}


def _launch_on(stream, dev: int, *tensors):
    """The raw stream handle of a call on ``stream`` (the current one if None);
    refuses tensors that are not on device ``dev``, the current one, where the
    kernels run."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {t.device} and cuda:{dev}: needs all of them on one device")
    current = torch._C._cuda_getDevice()
    if dev != current or (stream is not None and stream.device.index != dev):
        raise ValueError(f"tensors on cuda:{dev}: needs that device to be the current one "
                         f"(cuda:{current}) and the stream's")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _want(t, dtype, shape, name):
    """_need, with the common case checked first."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _need(t, dtype, shape, name)


def _misfit(**sizes) -> str | None:
    """Names the first size that the library's 32-bit arguments cannot hold."""
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:
            return f"{name}={v}: needs a size of at most {2 ** 31 - 1}"
    return None


def _fits(**sizes) -> None:
    why = _misfit(**sizes)
    if why:
        raise ValueError(why)


def _new(shape, dtype, device, stream):
    """An output of a call on ``stream``, from that stream's memory."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def route(logits, top_k: int, bias=None, n_groups: int = 1, topk_groups: int = 1,
          score: str = "softmax", renormalize: bool = True, scale: float = 1.0, ids=None,
          weights=None, stream=None):
    """(ids int32 [m, top_k], weights FP32 [m, top_k]): the experts of each row
    of logits [m, n_experts] (BF16 or FP32), best first, ties to the lower
    index; ``bias`` (FP32 [n_experts]) is added to the scores for the choice
    only; ids are -1 where nothing is left to choose (sk_route)."""
    m, n = logits.shape
    if (m | n | top_k | n_groups | topk_groups) >> 31:  # any negative, or beyond 31 bits
        _fits(m=m, n_experts=n, top_k=top_k, n_groups=n_groups, topk_groups=topk_groups)
    bf16 = logits.dtype is torch.bfloat16
    _want(logits, torch.bfloat16 if bf16 else torch.float32, (m, n), "logits")
    if score not in SCORES:
        raise ValueError(f"score: {score!r}, needs one of {sorted(SCORES)}")
    if bias is not None:
        _want(bias, torch.float32, (n,), "bias")
    if ids is None:
        ids = _new((m, top_k), torch.int32, logits.device, stream)
    else:
        _want(ids, torch.int32, (m, top_k), "ids")
    if weights is None:
        weights = _new((m, top_k), torch.float32, logits.device, stream)
    else:
        _want(weights, torch.float32, (m, top_k), "weights")
    s = _launch_on(stream, logits.get_device(), bias, ids, weights)
    _check(lib().sk_route(logits.data_ptr(), 0 if bf16 else 1,
                          None if bias is None else bias.data_ptr(), ids.data_ptr(),
                          weights.data_ptr(), m, n, n_groups, topk_groups, top_k, SCORES[score],
                          1 if renormalize else 0, scale, s))
    return ids, weights


def int8_quantize(z, q=None, scale=None, stream=None):
    """(q int8 [m, n], scale FP32 [m]): int8 codes of BF16 z [m, n], one scale
    per row (amax / 127): m token rows, or the output features of a weight."""
    m, n = z.shape
    if (m | n) >> 31:
        _fits(m=m, n=n)
    _want(z, torch.bfloat16, (m, n), "z")
    if q is None:
        q = _new((m, n), torch.int8, z.device, stream)
    else:
        _want(q, torch.int8, (m, n), "q")
    if scale is None:
        scale = _new((m,), torch.float32, z.device, stream)
    else:
        _want(scale, torch.float32, (m,), "scale")
    s = _launch_on(stream, z.get_device(), q, scale)
    _check(lib().sk_int8_quantize(z.data_ptr(), q.data_ptr(), scale.data_ptr(), m, n, s))
    return q, scale


def gemm_int8_supported(m: int, n: int, k: int, splits: int = 0) -> str | None:
    """None if the int8 GEMM has a launch for the shape, else why."""
    why = _misfit(m=m, n=n, k=k, splits=splits)
    if why:
        return why
    st = lib().sk_gemm_int8_supported(m, n, k, splits)
    return None if st == SK_OK else last_error()


def gemm_int8(xq, x_scale, wq, w_scale, out=None, splits: int = 0, stream=None):
    """out[m, n] = bf16((xq[m, k] @ wq[n, k]^T) * x_scale[m] * w_scale[n]): int8
    codes, an exact integer sum, FP32 scales per token and output feature."""
    m, k = xq.shape
    n = wq.shape[0]
    if (m | n | k | splits) >> 31:
        _fits(m=m, n=n, k=k, splits=splits)
    _want(xq, torch.int8, (m, k), "xq")
    _want(x_scale, torch.float32, (m,), "x_scale")
    _want(wq, torch.int8, (n, k), "wq")
    _want(w_scale, torch.float32, (n,), "w_scale")
    if out is None:
        out = _new((m, n), torch.bfloat16, xq.device, stream)
    else:
        _want(out, torch.bfloat16, (m, n), "out")
    s = _launch_on(stream, xq.get_device(), x_scale, wq, w_scale, out)
    _check(lib().sk_gemm_int8(xq.data_ptr(), x_scale.data_ptr(), wq.data_ptr(), w_scale.data_ptr(),
                              out.data_ptr(), m, n, k, splits, s))
    return out


def experts_int8_workspace(m: int, top_k: int, hidden: int, inter: int) -> int:
    if _misfit(m=m, top_k=top_k, hidden=hidden, inter=inter):
        return 0
    return int(lib().sk_experts_int8_workspace(m, top_k, hidden, inter))


_experts_workspace = functools.lru_cache(maxsize=256)(experts_int8_workspace)


def experts_int8(xq, x_scale, w13, s13, w2, s2, ids, weights, out=None, workspace=None,
                 stream=None):
    """(out BF16 [m, hidden], workspace): the routed experts of each token,
    out = sum_j weights[:, j] * w2[e](silu(gate[e](x)) * up[e](x)), e = ids[:, j],
    with int8 codes: xq [m, hidden], w13 [n_experts, 2 inter, hidden] (gate rows,
    then up rows), w2 [n_experts, hidden, inter], their scales x_scale [m], s13
    [n_experts, 2 inter], s2 [n_experts, hidden]; ids and weights as from
    ``route``, ids outside 0..n_experts-1 left out (sk_experts_int8)."""
    m, hidden = xq.shape
    n_experts, _, inter = w2.shape
    top_k = ids.shape[1]
    if (m | n_experts | top_k | hidden | inter) >> 31:
        _fits(m=m, n_experts=n_experts, top_k=top_k, hidden=hidden, inter=inter)
    _want(xq, torch.int8, (m, hidden), "xq")
    _want(x_scale, torch.float32, (m,), "x_scale")
    _want(w13, torch.int8, (n_experts, 2 * inter, hidden), "w13")
    _want(s13, torch.float32, (n_experts, 2 * inter), "s13")
    _want(w2, torch.int8, (n_experts, hidden, inter), "w2")
    _want(s2, torch.float32, (n_experts, hidden), "s2")
    _want(ids, torch.int32, (m, top_k), "ids")
    _want(weights, torch.float32, (m, top_k), "weights")
    if out is None:
        out = _new((m, hidden), torch.bfloat16, xq.device, stream)
    else:
        _want(out, torch.bfloat16, (m, hidden), "out")
    if workspace is None:
        workspace = _new((_experts_workspace(m, top_k, hidden, inter),), torch.uint8, xq.device, stream)
    else:
        _want(workspace, torch.uint8, (workspace.numel(),), "workspace")
    s = _launch_on(stream, xq.get_device(), x_scale, w13, s13, w2, s2, ids, weights, out, workspace)
    _check(lib().sk_experts_int8(
        xq.data_ptr(), x_scale.data_ptr(), w13.data_ptr(), s13.data_ptr(), w2.data_ptr(),
        s2.data_ptr(), ids.data_ptr(), weights.data_ptr(), out.data_ptr(), workspace.data_ptr(),
        workspace.numel(), m, n_experts, top_k, hidden, inter, s))
    return out, workspace


# ------------------------------------------- key/value cache held in 4 bits ----
MAX_CACHE_ROWS = 4096


def kv_block_bytes(page_size: int, head_dim: int) -> int:
    """Bytes of a KV head's part of a page (page_size 16, 32 or 64 tokens,
    head_dim 64 or 128): the last dimension of a cache."""
    if _misfit(page_size=page_size, head_dim=head_dim):
        return 0
    return int(lib().sk_kv_block_bytes(page_size, head_dim))


def _token_stride(x, name):
    """Values from a token of x [b, t, heads, d] to the next: the tokens' rows may
    be parts of longer ones."""
    b, t, heads, d = x.shape
    sb, st, sh, sd = x.stride()
    step = st if t > 1 else sb if b > 1 else heads * d
    if not x.is_cuda or sd != 1 or (heads > 1 and sh != d) or (b > 1 and t > 1 and sb != t * st):
        raise ValueError(f"{name}: needs a CUDA tensor of contiguous token rows a fixed stride apart")
    return step


def _sizes(t, dims, name):
    """The shape of t, which has that many dimensions."""
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name}: shape {tuple(shape)}, needs {dims} dimensions")
    return shape


def _layer_sizes(cache, table, page_size, head_dim, b, t):
    """(pages, kv_heads, width) of a layer's cache uint8 [pages, kv_heads, block] and
    the table int32 [b, width]."""
    pages, heads, _ = _sizes(cache, 3, "cache")
    _, width = _sizes(table, 2, "table")
    if (b | t | pages | heads | width | page_size) >> 31:
        _fits(b=b, t=t, pages=pages, kv_heads=heads, width=width, page_size=page_size)
    _want(cache, torch.uint8, (pages, heads, page_size * head_dim * 9 // 8), "cache")
    _want(table, torch.int32, (b, width), "table")
    return pages, heads, width


def kv_append(k, v, k_global_scale, v_global_scale, cache, table, lens, page_size: int, stream=None,
              new_lens=None, fresh=None):
    """Quantizes the last t tokens of each row, k and v BF16 [b, t, kv_heads, d], into
    a layer's cache uint8 [pages, kv_heads, block], in place: token j of row i at
    position lens[i] - t + j of the pages that table int32 [b, width] names. k and v
    may be parts of longer rows (sk_kv_append). With ``new_lens`` int32 [b], what kv_resize
    was given, rows that it refused or that wait are left out; with ``fresh`` int32 [b] row i
    brings its last fresh[i] tokens alone (sk_kv_append_ex)."""
    b, t, heads, d = _sizes(k, 4, "k")
    if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16:
        raise ValueError(f"k, v: dtypes {k.dtype}, {v.dtype}, need torch.bfloat16")
    if v.shape != k.shape:
        raise ValueError(f"v: shape {tuple(v.shape)}, needs {tuple(k.shape)}")
    ks, vs = _token_stride(k, "k"), _token_stride(v, "v")
    pages, kv_heads, width = _layer_sizes(cache, table, page_size, d, b, t)
    if kv_heads != heads:
        raise ValueError(f"k: {heads} heads, needs the cache's {kv_heads}")
    _want(k_global_scale, torch.float32, (1,), "k_global_scale")
    _want(v_global_scale, torch.float32, (1,), "v_global_scale")
    _want(lens, torch.int32, (b,), "lens")
    if new_lens is not None:
        _want(new_lens, torch.int32, (b,), "new_lens")
    if fresh is not None:
        _want(fresh, torch.int32, (b,), "fresh")
    s = _launch_on(stream, k.get_device(), v, k_global_scale, v_global_scale, cache, table, lens, new_lens,
                   fresh)
    _check(lib().sk_kv_append_ex(k.data_ptr(), v.data_ptr(), k_global_scale.data_ptr(),
                                 v_global_scale.data_ptr(), cache.data_ptr(), table.data_ptr(),
                                 lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(),
                                 None if fresh is None else fresh.data_ptr(), b, t, heads, d, page_size,
                                 pages, width, ks, vs, s))


def attn_nvfp4_workspace(b: int, t: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    if _misfit(b=b, t=t, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim):
        return 0
    return int(lib().sk_attn_nvfp4_workspace(b, t, q_heads, kv_heads, head_dim))


_attn_workspace = functools.lru_cache(maxsize=256)(attn_nvfp4_workspace)


def attn_nvfp4(q, k_global_scale, v_global_scale, cache, table, lens, page_size: int, scale=None,
               window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """(out BF16 [b, t, q_heads, d], lse, workspace): attention of the last t tokens of
    each row, q BF16 [b, t, q_heads, d], over a layer's cache uint8 [pages, kv_heads,
    block]; token j of row i sees the keys up to its position lens[i] - t + j, with
    ``window`` the last that many of them. ``scale`` is 1 / sqrt(d) if None; ``lse``
    (FP32 [b, t, q_heads]) may be a tensor, True (allocate) or None (not stored)
    (sk_attn_nvfp4)."""
    b, t, heads, d = _sizes(q, 4, "q")
    if q.dtype is not torch.bfloat16:
        raise ValueError(f"q: dtype {q.dtype}, needs torch.bfloat16")
    stride = _token_stride(q, "q")
    if window >> 31:
        _fits(window=window)
    pages, kv_heads, width = _layer_sizes(cache, table, page_size, d, b, t)
    _want(k_global_scale, torch.float32, (1,), "k_global_scale")
    _want(v_global_scale, torch.float32, (1,), "v_global_scale")
    _want(lens, torch.int32, (b,), "lens")
    if out is None:
        out = _new((b, t, heads, d), torch.bfloat16, q.device, stream)
    else:
        _want(out, torch.bfloat16, (b, t, heads, d), "out")
    if lse is True:
        lse = _new((b, t, heads), torch.float32, q.device, stream)
    elif lse is not None:
        _want(lse, torch.float32, (b, t, heads), "lse")
    if workspace is None:
        workspace = _new((_attn_workspace(b, t, heads, kv_heads, d),), torch.uint8, q.device, stream)
    else:
        _want(workspace, torch.uint8, (workspace.numel(),), "workspace")
    s = _launch_on(stream, q.get_device(), k_global_scale, v_global_scale, cache, table, lens, out, lse,
                   workspace)
    _check(lib().sk_attn_nvfp4(
        q.data_ptr(), k_global_scale.data_ptr(), v_global_scale.data_ptr(), cache.data_ptr(),
        table.data_ptr(), lens.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.numel(), b, t, heads, kv_heads, d, page_size, pages, width,
        stride, d ** -0.5 if scale is None else scale, window, s))
    return out, lse, workspace


def kv_resize_workspace(rows: int, pages: int) -> int:
    if _misfit(rows=rows, pages=pages):
        return 0
    return int(lib().sk_kv_resize_workspace(rows, pages))


def kv_compact_workspace(pages: int) -> int:
    if _misfit(pages=pages):
        return 0
    return int(lib().sk_kv_compact_workspace(pages))


def _pages_sizes(cache, table, lens, refs, page_size):
    """(layers, pages, kv_heads, head_dim, rows, width) of a cache's bookkeeping."""
    layers, pages, heads, block = _sizes(cache, 4, "cache")
    rows, width = _sizes(table, 2, "table")
    if (layers | pages | heads | rows | width | page_size) >> 31:
        _fits(layers=layers, pages=pages, kv_heads=heads, rows=rows, width=width, page_size=page_size)
    d = block * 8 // (9 * page_size) if page_size > 0 else 0
    if page_size > 0 and d * page_size * 9 != block * 8:
        raise ValueError(f"cache: blocks of {block} bytes, not of {page_size} tokens")
    _want(cache, torch.uint8, (layers, pages, heads, block), "cache")
    _want_pages(table, lens, refs, pages, rows, width)
    return layers, pages, heads, d, rows, width


def _want_pages(table, lens, refs, pages, rows, width):
    _want(table, torch.int32, (rows, width), "table")
    _want(lens, torch.int32, (rows,), "lens")
    _want(refs, torch.int32, (pages,), "refs")


def kv_resize(new_lens, cache, table, lens, refs, page_size: int, status=None, workspace=None,
              stream=None):
    """(status int32 [rows], workspace): gives each row of table int32 [rows, width] the
    length new_lens[i] (negative: as it is), adding pages from the free ones or giving
    them back; a partly filled last page that others hold too is copied first, in all
    layers of cache uint8 [layers, pages, kv_heads, block]. table, lens and refs int32
    [pages] (how many rows hold a page) are updated in place; status is 1 for a row
    refused for want of pages, 2 for a length out of range (sk_kv_resize)."""
    layers, pages, heads, d, rows, width = _pages_sizes(cache, table, lens, refs, page_size)
    _want(new_lens, torch.int32, (rows,), "new_lens")
    if status is None:
        status = _new((rows,), torch.int32, table.device, stream)
    else:
        _want(status, torch.int32, (rows,), "status")
    if workspace is None:
        workspace = _new((_resize_workspace(rows, pages),), torch.uint8, table.device, stream)
    else:
        _want(workspace, torch.uint8, (workspace.numel(),), "workspace")
    s = _launch_on(stream, table.get_device(), new_lens, cache, lens, refs, status, workspace)
    _check(lib().sk_kv_resize(new_lens.data_ptr(), cache.data_ptr(), table.data_ptr(), lens.data_ptr(),
                              refs.data_ptr(), status.data_ptr(), workspace.data_ptr(),
                              workspace.numel(), rows, width, pages, layers, heads, d, page_size, s))
    return status, workspace


_resize_workspace = functools.lru_cache(maxsize=256)(kv_resize_workspace)
_compact_workspace = functools.lru_cache(maxsize=256)(kv_compact_workspace)


def kv_fork(parents, table, lens, refs, page_size: int, status=None, stream=None):
    """status int32 [rows]: row i of table becomes what row parents[i] was before the
    call (negative, or i: as it is); the rows share their pages. table, lens and refs are
    updated in place; status is 2 for a parent that is no row (sk_kv_fork)."""
    rows, width = _sizes(table, 2, "table")
    pages, = _sizes(refs, 1, "refs")
    if (rows | width | pages | page_size) >> 31:
        _fits(rows=rows, width=width, pages=pages, page_size=page_size)
    _want_pages(table, lens, refs, pages, rows, width)
    _want(parents, torch.int32, (rows,), "parents")
    if status is None:
        status = _new((rows,), torch.int32, table.device, stream)
    else:
        _want(status, torch.int32, (rows,), "status")
    s = _launch_on(stream, table.get_device(), parents, lens, refs, status)
    _check(lib().sk_kv_fork(parents.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                            status.data_ptr(), rows, width, pages, page_size, s))
    return status


def kv_compact(cache, table, lens, refs, page_size: int, page_map=None, workspace=None, stream=None):
    """(page_map int32 [pages], workspace): moves the pages in use to the lowest numbers, in
    all layers of cache uint8 [layers, pages, kv_heads, block]; table and refs follow, in
    place. page_map is the new number of each page, -1 of a free one (sk_kv_compact)."""
    layers, pages, heads, d, rows, width = _pages_sizes(cache, table, lens, refs, page_size)
    if page_map is None:
        page_map = _new((pages,), torch.int32, table.device, stream)
    else:
        _want(page_map, torch.int32, (pages,), "page_map")
    if workspace is None:
        workspace = _new((_compact_workspace(pages),), torch.uint8, table.device, stream)
    else:
        _want(workspace, torch.uint8, (workspace.numel(),), "workspace")
    s = _launch_on(stream, table.get_device(), cache, lens, refs, page_map, workspace)
    _check(lib().sk_kv_compact(cache.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                               page_map.data_ptr(), workspace.data_ptr(), workspace.numel(), rows,
                               width, pages, layers, heads, d, page_size, s))
    return page_map, workspace


# ----------------------------------------------------------- diagnostics ----
def device_status(clear: bool = True) -> int:
    """The device status word (OR of SK_DEVICE_WAIT_* bits); synchronizes."""
    v = ctypes.c_uint32(0)
    _check(lib().sk_device_status(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


SK_DEVICE_WAIT_PROBE = 0x10


def wait_probe(limit_us: int, stream=None) -> None:
    """Launches a kernel whose bounded wait is meant to run out after limit_us
    microseconds; it sets SK_DEVICE_WAIT_PROBE in the device status word."""
    _check(lib().sk_wait_probe(limit_us, _stream(stream)))


def convert_probe(kind: int, inp: torch.Tensor, stream=None) -> torch.Tensor:
    """Runs one device format conversion over ``inp`` (see sk_convert_probe)."""
    n = inp.numel()
    if kind == 3:
        _need(inp, torch.uint8, (n,), "inp")
        out = torch.empty(n, dtype=torch.float32, device=inp.device)
    else:
        _need(inp, torch.float32, (n,), "inp")
        out = torch.empty(n, dtype=torch.int16 if kind == 2 else torch.uint8, device=inp.device)
    _check(lib().sk_convert_probe(kind, _ptr(inp), _ptr(out), n, _stream(stream)))
    return out
