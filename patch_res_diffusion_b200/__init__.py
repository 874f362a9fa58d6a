"""B200 (sm_100a) patch-restricted self-attention: Python binding.

A thin ctypes layer over the C ABI in ``include/npa.h`` (``libnpa_b200.so``,
built in-tree by ``patch_res_diffusion_b200.build``). The functions below carry
the C names and only marshal arguments; every step of the computation runs in
the library's CUDA kernels. There is no fallback: if the library is missing or
a call fails, an exception is raised.

* ``npa_attention_fwd`` - Neighborhood Patch Attention (ScaleDiff summary,
  "Approach"): non-overlapping query patches, each attending to its patch
  grown by a margin and clipped to the grid.
* ``pcpp_attention_fwd`` - partially conditioned attention (PCPP review, "What
  carries the argument"): row strips attending to themselves plus the nearest
  ceil(p * rows) rows of each adjacent strip.
* ``pcpp_attention_fwd_stale`` - PCPP as it runs across devices (PCPP review,
  "Core claim"): the strip's own keys from the current step, the borrowed
  neighbour rows from the previous step's keys/values.
* ``npa_global_query_attention_fwd`` (and ``..._noalloc``) - the text-query
  half of joint attention: global tokens as queries over all keys.
* ``npa_multidiffusion_attention_fwd`` - the overlapping-window comparator
  (ScaleDiff summary, "Approach": MultiDiffusion averages overlapping
  patches): each NPA window attends within itself and a token's output is the
  mean over the windows that contain it.
* ``asg_guidance_combine`` - asynchronous structure guidance (ASGDiffusion
  review, "core_discovery"): eps + w_t * M * (eps_ref - eps) per patch.
* ``npa_cross_attention_fwd`` - cross attention of image tokens (or a few
  latent queries) to an encoder's states of another length.
* ``npa_kv8_store`` and ``npa_kv8_cross_attention_fwd`` - a key/value cache in
  e4m3 with a power-of-two scale per 64 tokens and head, and the attention
  over it.
* ``npa_group_norm_act`` - group norm with an activation, channels last.

The lower-case helpers (``npa_attention``, ``pcpp_attention``,
``pcpp_attention_stale``, ``global_query_attention``,
``multidiffusion_attention``, ``asg_combine``, ``cross_attention``,
``kv8_store``, ``kv8_cross_attention``, ``group_norm``) take torch CUDA tensors
and allocate outputs and workspaces; the computation is the same C call.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
from typing import Optional

__all__ = [
    "NpaError", "lib", "LIB_PATH", "NPA_OK", "NPA_ERR_INVALID_ARG", "NPA_ERR_UNSUPPORTED",
    "NPA_ERR_MISALIGNED", "NPA_ERR_CUDA", "NPA_ERR_DEVICE_TIMEOUT", "npa_attention_fwd",
    "pcpp_attention_fwd", "pcpp_neighbor_rows", "npa_useful_flops", "pcpp_useful_flops",
    "npa_device_status", "npa_selftest_wait_timeout", "npa_status_string", "npa_attention",
    "pcpp_attention", "pcpp_attention_fwd_stale", "pcpp_attention_stale", "npa_global_query_attention_fwd",
    "npa_global_query_workspace_size", "npa_global_query_attention_fwd_noalloc", "global_query_attention",
    "npa_multidiffusion_attention_fwd", "npa_multidiffusion_workspace_size", "npa_multidiffusion_useful_flops",
    "multidiffusion_attention", "asg_guidance_combine", "asg_combine", "EXPORTED_SYMBOLS", "DEBUG_LIB_PATH",
    "DEBUG_ONLY_SYMBOLS", "NPA_ERR_DEVICE_BOUNDS", "use_bounds_checking", "npa_debug_withhold_arrival_once",
    "NPA_DTYPE_BF16", "NPA_DTYPE_FP16", "NPA_DTYPE_FP32", "NPA_ACT_NONE", "NPA_ACT_SILU", "KV8_BLOCK", "Kv8Cache",
    "npa_cross_attention_fwd", "npa_cross_attention_workspace_size", "npa_kv8_store", "npa_kv8_cross_attention_fwd",
    "npa_group_norm_act", "npa_group_norm_workspace_size", "npa_device_ready", "cross_attention", "kv8_store",
    "kv8_cross_attention", "group_norm",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnpa_b200.so")
DEBUG_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnpa_b200_debug.so")

NPA_OK = 0
NPA_ERR_INVALID_ARG = 1
NPA_ERR_UNSUPPORTED = 2
NPA_ERR_MISALIGNED = 3
NPA_ERR_CUDA = 4
NPA_ERR_DEVICE_TIMEOUT = 5
NPA_ERR_DEVICE_BOUNDS = 6

NPA_DTYPE_BF16 = 0
NPA_DTYPE_FP16 = 1
NPA_DTYPE_FP32 = 2
NPA_ACT_NONE = 0
NPA_ACT_SILU = 1
KV8_BLOCK = 64  # tokens of one head that share a scale of the 8-bit cache

EXPORTED_SYMBOLS = (
    "npa_attention_fwd", "pcpp_attention_fwd", "pcpp_attention_fwd_stale", "pcpp_neighbor_rows", "npa_useful_flops",
    "pcpp_useful_flops", "npa_device_status", "npa_selftest_wait_timeout", "npa_status_string",
    "npa_global_query_attention_fwd", "npa_global_query_workspace_size",
    "npa_global_query_attention_fwd_noalloc", "npa_multidiffusion_attention_fwd",
    "npa_multidiffusion_workspace_size", "npa_multidiffusion_useful_flops", "asg_guidance_combine",
    "npa_cross_attention_fwd", "npa_cross_attention_workspace_size", "npa_kv8_store", "npa_kv8_cross_attention_fwd",
    "npa_group_norm_act", "npa_group_norm_workspace_size", "npa_device_ready",
)
# exported by the bounds-checking build only
DEBUG_ONLY_SYMBOLS = ("npa_debug_withhold_arrival_once",)


class NpaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {npa_status_string(code)} ({code})")
        self.code = code


class _GlobalKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_tokens", ctypes.c_int)]


class _Strides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("token", ctypes.c_int64)]


class _Kv8Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("capacity", ctypes.c_int)]


_LIB: Optional[ctypes.CDLL] = None
_LOADED = {}


def lib() -> ctypes.CDLL:
    """The C library in use (the normal build unless use_bounds_checking(True)
    switched to the bounds-checking one). Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        _LIB = _load(LIB_PATH)
    return _LIB


def use_bounds_checking(on: bool) -> None:
    """Routes every call of this module to the bounds-checking build
    (``libnpa_b200_debug.so``: device-side checks of every TMA box origin and
    output row, NPA_ERR_DEVICE_BOUNDS on a failure) or back to the normal one.
    Each library keeps its own device status word."""
    global _LIB
    _LIB = _load(DEBUG_LIB_PATH if on else LIB_PATH)


def _load(path: str) -> ctypes.CDLL:
    if path not in _LOADED:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python -m patch_res_diffusion_b200.build`")
        L = ctypes.CDLL(path)
        vp, i, d = ctypes.c_void_p, ctypes.c_int, ctypes.c_double
        gkv = ctypes.POINTER(_GlobalKV)
        L.npa_attention_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, gkv, vp]
        L.npa_attention_fwd.restype = i
        L.pcpp_attention_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, d, gkv, vp]
        L.pcpp_attention_fwd.restype = i
        L.pcpp_attention_fwd_stale.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, d, i, i, gkv, vp]
        L.pcpp_attention_fwd_stale.restype = i
        L.npa_global_query_attention_fwd.argtypes = [vp] * 6 + [i] * 6 + [vp, ctypes.c_size_t, vp]
        L.npa_global_query_attention_fwd.restype = i
        L.npa_global_query_attention_fwd_noalloc.argtypes = [vp] * 6 + [i] * 6 + [vp]
        L.npa_global_query_attention_fwd_noalloc.restype = i
        L.npa_multidiffusion_attention_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, gkv, vp,
                                                       ctypes.c_size_t, vp]
        L.npa_multidiffusion_attention_fwd.restype = i
        L.npa_multidiffusion_workspace_size.argtypes = [i] * 7
        L.npa_multidiffusion_workspace_size.restype = ctypes.c_size_t
        L.npa_multidiffusion_useful_flops.argtypes = [i] * 8
        L.npa_multidiffusion_useful_flops.restype = d
        L.asg_guidance_combine.argtypes = [vp] * 4 + [i] * 4 + [ctypes.c_float, vp]
        L.asg_guidance_combine.restype = i
        st, kv8, f = ctypes.POINTER(_Strides), ctypes.POINTER(_Kv8Cache), ctypes.c_float
        L.npa_cross_attention_fwd.argtypes = [vp] * 4 + [i] * 7 + [st] * 4 + [vp, vp, f, vp, ctypes.c_size_t, vp]
        L.npa_cross_attention_fwd.restype = i
        L.npa_device_ready.argtypes = []
        L.npa_device_ready.restype = i
        L.npa_cross_attention_workspace_size.argtypes = [i] * 6
        L.npa_cross_attention_workspace_size.restype = ctypes.c_size_t
        L.npa_kv8_store.argtypes = [vp, vp, kv8] + [i] * 5 + [vp, i, st, st, vp]
        L.npa_kv8_store.restype = i
        L.npa_kv8_cross_attention_fwd.argtypes = [vp, kv8, vp] + [i] * 6 + [st, st, vp, vp, f, vp, ctypes.c_size_t, vp]
        L.npa_kv8_cross_attention_fwd.restype = i
        L.npa_group_norm_act.argtypes = [vp] * 4 + [i] * 6 + [ctypes.c_int64] * 4 + [f, i, vp, ctypes.c_size_t, vp]
        L.npa_group_norm_act.restype = i
        L.npa_group_norm_workspace_size.argtypes = [i] * 5
        L.npa_group_norm_workspace_size.restype = ctypes.c_size_t
        L.npa_global_query_workspace_size.argtypes = [i] * 6
        L.npa_global_query_workspace_size.restype = ctypes.c_size_t
        L.pcpp_neighbor_rows.argtypes = [i, d]
        L.pcpp_neighbor_rows.restype = i
        L.npa_useful_flops.argtypes = [i, i, i, i, i, i, i, i]
        L.npa_useful_flops.restype = d
        L.pcpp_useful_flops.argtypes = [i, i, i, i, i, i, d, i]
        L.pcpp_useful_flops.restype = d
        L.npa_device_status.argtypes = [vp]
        L.npa_device_status.restype = i
        L.npa_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
        L.npa_selftest_wait_timeout.restype = i
        L.npa_status_string.argtypes = [i]
        L.npa_status_string.restype = ctypes.c_char_p
        if path == DEBUG_LIB_PATH:
            L.npa_debug_withhold_arrival_once.argtypes = [ctypes.c_uint32]
            L.npa_debug_withhold_arrival_once.restype = i
        _LOADED[path] = L
    return _LOADED[path]


def _ptr(x) -> Optional[int]:
    """Device address of a tensor (``data_ptr``) or a raw integer address."""
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    return int(x)


def _stream(stream) -> Optional[int]:
    if stream is None:
        try:
            import torch
            if torch.cuda.is_initialized() or torch.cuda.is_available():
                return _raw_stream_of()(torch.cuda.current_device())
        except ImportError:
            pass
        return None
    if hasattr(stream, "cuda_stream"):
        return int(stream.cuda_stream)
    return int(stream)


def _gkv(global_k, global_v, n_tokens: int):
    if not n_tokens:
        return None
    return ctypes.byref(_GlobalKV(_ptr(global_k), _ptr(global_v), int(n_tokens)))


def _check(code: int, what: str) -> None:
    if code != NPA_OK:
        raise NpaError(code, what)


def npa_attention_fwd(q, k, v, o, B: int, heads: int, H: int, W: int, d: int, patch: int, margin: int,
                      global_k=None, global_v=None, n_global: int = 0, stream=None) -> None:
    """C ``npa_attention_fwd``: bf16 [B, heads, H*W, d] device buffers."""
    _check(lib().npa_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, heads, H, W, d, patch, margin,
                                   _gkv(global_k, global_v, n_global), _stream(stream)),
           "npa_attention_fwd")


def pcpp_attention_fwd(q, k, v, o, B: int, heads: int, H: int, W: int, d: int, n_strips: int, p: float,
                       global_k=None, global_v=None, n_global: int = 0, stream=None) -> None:
    """C ``pcpp_attention_fwd``: bf16 [B, heads, H*W, d] device buffers."""
    _check(lib().pcpp_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, heads, H, W, d, n_strips,
                                    float(p), _gkv(global_k, global_v, n_global), _stream(stream)),
           "pcpp_attention_fwd")


def pcpp_attention_fwd_stale(q, k, v, k_stale, v_stale, o, B: int, heads: int, H: int, W: int, d: int,
                             n_strips: int, p: float, strip_begin: int, strip_count: int, global_k=None,
                             global_v=None, n_global: int = 0, stream=None) -> None:
    """C ``pcpp_attention_fwd_stale``: own-strip keys from k/v, borrowed rows from k_stale/v_stale."""
    _check(lib().pcpp_attention_fwd_stale(_ptr(q), _ptr(k), _ptr(v), _ptr(k_stale), _ptr(v_stale), _ptr(o), B,
                                          heads, H, W, d, n_strips, float(p), strip_begin, strip_count,
                                          _gkv(global_k, global_v, n_global), _stream(stream)),
           "pcpp_attention_fwd_stale")


def npa_global_query_attention_fwd(gq, k, v, gk, gv, go, B: int, heads: int, H: int, W: int, d: int, G: int,
                                   workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    """C ``npa_global_query_attention_fwd``: global-token queries over all keys."""
    _check(lib().npa_global_query_attention_fwd(_ptr(gq), _ptr(k), _ptr(v), _ptr(gk), _ptr(gv), _ptr(go), B, heads,
                                                H, W, d, G, _ptr(workspace), int(workspace_bytes),
                                                _stream(stream)),
           "npa_global_query_attention_fwd")


def npa_global_query_attention_fwd_noalloc(gq, k, v, gk, gv, go, B: int, heads: int, H: int, W: int, d: int,
                                           G: int, stream=None) -> None:
    """C ``npa_global_query_attention_fwd_noalloc``: the same computation with
    the split partials in the library's fixed device array (no caller memory)."""
    _check(lib().npa_global_query_attention_fwd_noalloc(_ptr(gq), _ptr(k), _ptr(v), _ptr(gk), _ptr(gv), _ptr(go),
                                                        B, heads, H, W, d, G, _stream(stream)),
           "npa_global_query_attention_fwd_noalloc")


def npa_multidiffusion_attention_fwd(q, k, v, o, B: int, heads: int, H: int, W: int, d: int, patch: int,
                                     margin: int, workspace, workspace_bytes: int, global_k=None, global_v=None,
                                     n_global: int = 0, stream=None) -> None:
    """C ``npa_multidiffusion_attention_fwd``: overlapping-window attention;
    ``workspace`` holds npa_multidiffusion_workspace_size() bytes."""
    _check(lib().npa_multidiffusion_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, heads, H, W, d, patch,
                                                  margin, _gkv(global_k, global_v, n_global), _ptr(workspace),
                                                  int(workspace_bytes), _stream(stream)),
           "npa_multidiffusion_attention_fwd")


def npa_multidiffusion_workspace_size(B, heads, H, W, d, patch, margin) -> int:
    return int(lib().npa_multidiffusion_workspace_size(B, heads, H, W, d, patch, margin))


def npa_multidiffusion_useful_flops(B, heads, H, W, d, patch, margin, G=0) -> float:
    return float(lib().npa_multidiffusion_useful_flops(B, heads, H, W, d, patch, margin, G))


def asg_guidance_combine(eps, eps_ref, mask, out, n_patches: int, B: int, C: int, S: int, w_t: float,
                         stream=None) -> None:
    """C ``asg_guidance_combine``: out = eps + w_t * mask * (eps_ref - eps)."""
    _check(lib().asg_guidance_combine(_ptr(eps), _ptr(eps_ref), _ptr(mask), _ptr(out), n_patches, B, C, S,
                                      float(w_t), _stream(stream)),
           "asg_guidance_combine")


@functools.lru_cache(maxsize=1024)
def _strides(s):
    """None (contiguous) or a tuple of (batch, head, token) strides in elements."""
    return None if s is None else ctypes.byref(_Strides(*s))


@functools.lru_cache(maxsize=None)
def _raw_stream_of():
    """A function from a device index to its current stream's handle (torch's
    cheap query of it where this version has one)."""
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream",
                   lambda index: int(torch.cuda.current_stream(index).cuda_stream))


def npa_cross_attention_fwd(q, k, v, o, dtype: int, B: int, heads: int, kv_heads: int, Lq: int, Lk: int, d: int,
                            q_strides=None, k_strides=None, v_strides=None, o_strides=None, kv_lens=None,
                            key_mask=None, scale: float = 0.0, workspace=None, workspace_bytes: int = 0,
                            stream=None) -> None:
    """C ``npa_cross_attention_fwd``: q, o [B, heads, Lq, d], k, v [B, kv_heads, Lk, d]; strides are (batch, head,
    token) in elements, None for contiguous."""
    _check(lib().npa_cross_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), dtype, B, heads, kv_heads, Lq, Lk, d,
                                         _strides(q_strides), _strides(k_strides), _strides(v_strides),
                                         _strides(o_strides), _ptr(kv_lens), _ptr(key_mask), scale, _ptr(workspace),
                                         int(workspace_bytes), _stream(stream)),
           "npa_cross_attention_fwd")


def npa_device_ready() -> None:
    """C ``npa_device_ready``: raises unless the current device runs this library."""
    _check(lib().npa_device_ready(), "npa_device_ready")


def npa_cross_attention_workspace_size(B, heads, kv_heads, Lq, Lk, d) -> int:
    return int(lib().npa_cross_attention_workspace_size(B, heads, kv_heads, Lq, Lk, d))


def npa_kv8_store(k, v, cache_k, cache_v, k_scale, v_scale, capacity: int, dtype: int, B: int, kv_heads: int, d: int,
                  start: int, n_tokens: int, starts=None, k_strides=None, v_strides=None, stream=None) -> None:
    """C ``npa_kv8_store``: k, v [B, kv_heads, n_tokens, d] into the cache's codes and scales."""
    c = _Kv8Cache(_ptr(cache_k), _ptr(cache_v), _ptr(k_scale), _ptr(v_scale), capacity)
    _check(lib().npa_kv8_store(_ptr(k), _ptr(v), ctypes.byref(c), dtype, B, kv_heads, d, start, _ptr(starts),
                               n_tokens, _strides(k_strides), _strides(v_strides), _stream(stream)),
           "npa_kv8_store")


def npa_kv8_cross_attention_fwd(q, cache_k, cache_v, k_scale, v_scale, capacity: int, o, B: int, heads: int,
                                kv_heads: int, Lq: int, Lk: int, d: int, q_strides=None, o_strides=None, kv_lens=None,
                                key_mask=None, scale: float = 0.0, workspace=None, workspace_bytes: int = 0,
                                stream=None) -> None:
    """C ``npa_kv8_cross_attention_fwd``: bf16 q, o over the first Lk tokens of an 8-bit cache."""
    c = _Kv8Cache(_ptr(cache_k), _ptr(cache_v), _ptr(k_scale), _ptr(v_scale), capacity)
    _check(lib().npa_kv8_cross_attention_fwd(_ptr(q), ctypes.byref(c), _ptr(o), B, heads, kv_heads, Lq, Lk, d,
                                             _strides(q_strides), _strides(o_strides), _ptr(kv_lens), _ptr(key_mask),
                                             scale, _ptr(workspace), int(workspace_bytes), _stream(stream)),
           "npa_kv8_cross_attention_fwd")


def npa_group_norm_act(x, weight, bias, y, dtype: int, weight_dtype: int, B: int, N: int, C: int, groups: int,
                       x_batch_stride: int, x_token_stride: int, y_batch_stride: int, y_token_stride: int, eps: float,
                       act: int, workspace, workspace_bytes: int, stream=None) -> None:
    """C ``npa_group_norm_act``: x, y [B, N, C], statistics over the tokens and channels of a group."""
    _check(lib().npa_group_norm_act(_ptr(x), _ptr(weight), _ptr(bias), _ptr(y), dtype, weight_dtype, B, N, C, groups,
                                    x_batch_stride, x_token_stride, y_batch_stride, y_token_stride, eps, act,
                                    _ptr(workspace), int(workspace_bytes), _stream(stream)),
           "npa_group_norm_act")


def npa_group_norm_workspace_size(dtype, B, N, C, groups) -> int:
    return int(lib().npa_group_norm_workspace_size(dtype, B, N, C, groups))


def npa_global_query_workspace_size(B, heads, H, W, d, G) -> int:
    return int(lib().npa_global_query_workspace_size(B, heads, H, W, d, G))


def pcpp_neighbor_rows(strip_rows: int, p: float) -> int:
    return int(lib().pcpp_neighbor_rows(strip_rows, float(p)))


def npa_useful_flops(B, heads, H, W, d, patch, margin, G=0) -> float:
    return float(lib().npa_useful_flops(B, heads, H, W, d, patch, margin, G))


def pcpp_useful_flops(B, heads, H, W, d, n_strips, p, G=0) -> float:
    return float(lib().pcpp_useful_flops(B, heads, H, W, d, n_strips, float(p), G))


def npa_device_status(stream=None) -> int:
    return int(lib().npa_device_status(_stream(stream)))


def npa_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _check(lib().npa_selftest_wait_timeout(int(limit_us), _stream(stream)), "npa_selftest_wait_timeout")


def npa_debug_withhold_arrival_once(wait_limit_us: int) -> None:
    """C ``npa_debug_withhold_arrival_once`` (bounds-checking build only):
    the next attention launch's first CTA withholds one arrival and its
    bounded waits of ``wait_limit_us`` run out (the abort path)."""
    L = lib()
    if not hasattr(L, "npa_debug_withhold_arrival_once"):
        raise NpaError(NPA_ERR_UNSUPPORTED, "npa_debug_withhold_arrival_once needs use_bounds_checking(True)")
    _check(L.npa_debug_withhold_arrival_once(int(wait_limit_us)), "npa_debug_withhold_arrival_once")


def npa_status_string(code: int) -> str:
    try:
        return lib().npa_status_string(int(code)).decode()
    except ImportError:
        return f"status {code}"


# ---------------------------------------------------------------------------
# torch conveniences (allocation of the output only; the call is the C one)
# ---------------------------------------------------------------------------

def _shape(q, H, W):
    if q.dim() != 4 or q.shape[2] != H * W:
        raise ValueError(f"expected [B, heads, H*W={H * W}, d], got {tuple(q.shape)}")
    return int(q.shape[0]), int(q.shape[1]), int(q.shape[3])


def npa_attention(q, k, v, H: int, W: int, patch: int, margin: int, global_k=None, global_v=None,
                  out=None, stream=None):
    """NPA forward on torch bf16 CUDA tensors [B, heads, H*W, d]; returns ``out``."""
    B, heads, d = _shape(q, H, W)
    if out is None:
        out = q.new_empty(q.shape)
    G = 0 if global_k is None else int(global_k.shape[2])
    npa_attention_fwd(q, k, v, out, B, heads, H, W, d, patch, margin, global_k, global_v, G, stream)
    return out


def pcpp_attention(q, k, v, H: int, W: int, n_strips: int, p: float, global_k=None, global_v=None,
                   out=None, stream=None):
    """PCPP forward on torch bf16 CUDA tensors [B, heads, H*W, d]; returns ``out``."""
    B, heads, d = _shape(q, H, W)
    if out is None:
        out = q.new_empty(q.shape)
    G = 0 if global_k is None else int(global_k.shape[2])
    pcpp_attention_fwd(q, k, v, out, B, heads, H, W, d, n_strips, p, global_k, global_v, G, stream)
    return out


def pcpp_attention_stale(q, k, v, k_stale, v_stale, H: int, W: int, n_strips: int, p: float, strips=None,
                         global_k=None, global_v=None, out=None, stream=None):
    """Two-source PCPP forward on torch bf16 CUDA tensors; ``strips`` is an
    optional (begin, count) range of strips to compute (default: all)."""
    B, heads, d = _shape(q, H, W)
    if out is None:
        out = q.new_empty(q.shape)
    begin, count = (0, n_strips) if strips is None else strips
    G = 0 if global_k is None else int(global_k.shape[2])
    pcpp_attention_fwd_stale(q, k, v, k_stale, v_stale, out, B, heads, H, W, d, n_strips, p, begin, count,
                             global_k, global_v, G, stream)
    return out


def global_query_attention(gq, k, v, gk, gv, H: int, W: int, out=None, split: bool = True, stream=None):
    """Global-token queries [B, heads, G, d] over all image and global keys
    (torch bf16 CUDA tensors); with ``split`` a workspace is allocated so the
    key range can be split across the GPU."""
    import torch
    B, heads, G, d = (int(x) for x in gq.shape)
    if out is None:
        out = gq.new_empty(gq.shape)
    ws, nbytes = None, 0
    if split:
        nbytes = npa_global_query_workspace_size(B, heads, H, W, d, G)
        if nbytes:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=gq.device)
    npa_global_query_attention_fwd(gq, k, v, gk, gv, out, B, heads, H, W, d, G, ws, nbytes, stream)
    return out


def multidiffusion_attention(q, k, v, H: int, W: int, patch: int, margin: int, global_k=None, global_v=None,
                             out=None, workspace=None, stream=None):
    """Overlapping-window attention on torch bf16 CUDA tensors [B, heads,
    H*W, d]; allocates the float32 window workspace unless one is given."""
    import torch
    B, heads, d = _shape(q, H, W)
    if out is None:
        out = q.new_empty(q.shape)
    nbytes = npa_multidiffusion_workspace_size(B, heads, H, W, d, patch, margin)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    G = 0 if global_k is None else int(global_k.shape[2])
    npa_multidiffusion_attention_fwd(q, k, v, out, B, heads, H, W, d, patch, margin, workspace,
                                     workspace.numel() * workspace.element_size(), global_k, global_v, G, stream)
    return out


def asg_combine(eps, eps_ref, mask, w_t: float, out=None, stream=None):
    """ASG combine on torch bf16 CUDA tensors: eps [n, B, C, S], eps_ref
    [B, C, S], mask [n, B, S]; ``out=eps`` works in place."""
    n, B, C, S = (int(x) for x in eps.shape)
    if out is None:
        out = eps.new_empty(eps.shape)
    asg_guidance_combine(eps, eps_ref, mask, out, n, B, C, S, w_t, stream)
    return out


# ---------------------------------------------------------------------------
# The steps around the self-attention. Some of these calls run for a few
# microseconds, so what a call's shapes, strides and types decide - the checks,
# the stride structures, the workspace's size - is worked out once for each
# combination (the lru_cache'd functions) and looked up afterwards. What is
# looked up by is made of plain numbers and types: a tensor given for a number
# hashes by its identity, whatever it holds by then.
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _dtype_codes():
    import torch
    return {torch.bfloat16: NPA_DTYPE_BF16, torch.float16: NPA_DTYPE_FP16, torch.float32: NPA_DTYPE_FP32}


def _dtype_code(dtype, allowed) -> int:
    code = _dtype_codes().get(dtype)
    if code not in allowed:
        raise ValueError(f"unsupported dtype {dtype}")
    return code


def _device_of(first, *others) -> int:
    """The index of the CUDA device that all the tensors (or None) are on."""
    index = first.get_device()
    if index < 0:
        raise ValueError(f"expected CUDA tensors, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    return index


def _run_on(index, stream, body, *args):
    """``body(*args, handle)`` with device ``index`` and, when given, ``stream``
    current, so that outputs and workspaces come from the stream that the call
    runs on; handle is that stream's."""
    import torch
    if stream is None and index == torch.cuda.current_device():
        return body(*args, _raw_stream_of()(index))
    if getattr(stream, "device_index", index) != index:
        raise ValueError(f"stream of device {stream.device_index}, tensors on device {index}")
    with torch.cuda.device(index):
        if stream is None:
            return body(*args, _raw_stream_of()(index))
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", index))
        with torch.cuda.stream(stream):
            return body(*args, int(stream.cuda_stream))


def _int32(name, n) -> int:
    """n as an int that the C call can take (ctypes would drop its upper bits)."""
    n = operator.index(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name}: {n} does not fit in 32 bits")
    return n


def _heads_strides(name, shape, strides, want):
    """Checks a [B, heads, L, d] tensor's layout; its strides for the C call."""
    if tuple(shape) != tuple(want):
        raise ValueError(f"{name}: expected {tuple(want)}, got {tuple(shape)}")
    if strides[3] != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return _strides(strides[:3])


def _kept_keys(kv_lens, key_mask, B, Lk):
    import torch
    if kv_lens is not None and (kv_lens.dtype != torch.int32 or kv_lens.shape != (B,) or not kv_lens.is_contiguous()):
        raise ValueError(f"kv_lens: expected a contiguous int32 tensor of {B} lengths")
    if key_mask is not None and (key_mask.dtype not in (torch.bool, torch.uint8) or key_mask.shape != (B, Lk) or
                                 not key_mask.is_contiguous()):
        raise ValueError(f"key_mask: expected a contiguous bool or uint8 tensor [{B}, {Lk}]")


def _scale(scale) -> float:
    if scale is None:
        return 0.0
    scale = ctypes.c_float(scale).value   # as the C call gets it, where 0 means the default
    if not 0 < scale < float("inf"):
        raise ValueError(f"scale must be positive and finite in float32, got {scale}")
    return scale


def _like_strides(shape, strides):
    """The strides, for the C call, that torch.empty_like gives a tensor of this layout."""
    import torch
    like = torch.empty_like(torch.empty_strided(shape, strides, dtype=torch.uint8, device="meta"))
    return _heads_strides("out", shape, like.stride(), shape)


def _empty_bytes(n, like):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=like.device) if n else None


def _planned_bytes(size, *args) -> int:
    """A workspace size on the current device that may be kept: the 0 of a
    device that could not be asked raises instead."""
    nbytes = size(*args)
    if not nbytes:
        npa_device_ready()
    return nbytes


@functools.lru_cache(maxsize=1024)
def _cross_plan(index, split, q_shape, q_strides, k_shape, k_strides, v_shape, v_strides, q_dtype, k_dtype, v_dtype):
    """(sizes, strides and a fresh output's strides for the C call, workspace bytes)."""
    if len(q_shape) != 4 or len(k_shape) != 4:
        raise ValueError(f"expected [B, heads, L, d], got {tuple(q_shape)} and {tuple(k_shape)}")
    B, heads, Lq, d = (_int32("q", n) for n in q_shape)
    kv_heads, Lk = (_int32("k", n) for n in k_shape[1:3])
    strides = (_heads_strides("q", q_shape, q_strides, q_shape),
               _heads_strides("k", k_shape, k_strides, (B, kv_heads, Lk, d)),
               _heads_strides("v", v_shape, v_strides, k_shape))
    code = _dtype_code(q_dtype, (NPA_DTYPE_BF16, NPA_DTYPE_FP16))
    if not q_dtype == k_dtype == v_dtype:
        raise ValueError("q, k and v must have one dtype")
    nbytes = 0
    if split and index >= 0:
        nbytes = _planned_bytes(npa_cross_attention_workspace_size, B, heads, kv_heads, Lq, Lk, d)   # on `index`
    return (code, B, heads, kv_heads, Lq, Lk, d), strides, _like_strides(q_shape, q_strides), nbytes


def cross_attention(q, k, v, kv_lens=None, key_mask=None, scale: Optional[float] = None, out=None, split: bool = True,
                    stream=None):
    """Cross attention on torch bf16 or fp16 CUDA tensors: q [B, heads, Lq, d],
    k and v [B, kv_heads, Lk, d], any strides that are multiples of 8 elements
    with the last axis contiguous (a projection's ``[B, L, heads, d]`` seen
    through ``transpose(1, 2)``). What ``kv_lens`` (int32 [B]) or ``key_mask``
    (bool or uint8 [B, Lk], true: attend) leave out does not reach the output;
    a row without keys gives zeros. Forward only: the result carries no
    gradient. ``scale`` defaults to 1/sqrt(d). With
    ``split`` a workspace is allocated so that the key range can be split
    across the GPU. Returns ``out`` (by default laid out like q)."""
    index = q.get_device()
    if index < 0:   # refused below, after the shapes' own faults
        return _cross_attention(index, q, k, v, kv_lens, key_mask, scale, out, split, 0)
    return _run_on(index, stream, _cross_attention, index, q, k, v, kv_lens, key_mask, scale, out, split)


def _cross_attention(index, q, k, v, kv_lens, key_mask, scale, out, split, handle):
    import torch
    sizes, strides, o_strides, nbytes = _cross_plan(index, bool(split), q.shape, q.stride(), k.shape, k.stride(), v.shape,
                                                    v.stride(), q.dtype, k.dtype, v.dtype)
    lens = mask = None
    if kv_lens is not None or key_mask is not None:
        _kept_keys(kv_lens, key_mask, sizes[1], sizes[5])
        lens, mask = _ptr(kv_lens), _ptr(key_mask)
    _device_of(q, k, v, kv_lens, key_mask, out)
    if out is None:
        out = torch.empty_like(q)
    else:
        if out.dtype != q.dtype:
            raise ValueError("out must have q's dtype")
        o_strides = _heads_strides("out", out.shape, out.stride(), q.shape)
    ws = _empty_bytes(nbytes, q)
    code = lib().npa_cross_attention_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), *sizes, *strides, o_strides, lens, mask, _scale(scale),
        ws.data_ptr() if nbytes else None, nbytes, handle)
    if code:
        raise NpaError(code, "npa_cross_attention_fwd")
    return out


class Kv8Cache:
    """Keys and values in 8 bits: e4m3 codes ``k``, ``v`` [B, kv_heads,
    capacity, d] (``torch.float8_e4m3fn`` or uint8) and float32 scales
    ``k_scale``, ``v_scale`` [B, kv_heads, capacity / 64], value = code *
    scale. ``Kv8Cache.empty`` allocates one; ``kv8_store`` writes it."""

    __slots__ = ("_tensors", "index")

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        if k.dim() != 4 or k.shape != v.shape or k.shape[2] % KV8_BLOCK:
            raise ValueError(f"expected codes [B, kv_heads, capacity, d] with capacity a multiple of {KV8_BLOCK}, "
                             f"got {tuple(k.shape)} and {tuple(v.shape)}")
        want = (k.shape[0], k.shape[1], k.shape[2] // KV8_BLOCK)
        for t in (k_scale, v_scale):
            if t.shape != want or t.dtype != torch.float32:
                raise ValueError(f"expected float32 scales {want}, got {t.dtype} {tuple(t.shape)}")
        for t in (k, v):
            if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise ValueError(f"expected e4m3 or uint8 codes, got {t.dtype}")
        if not (k.is_contiguous() and v.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()):
            raise ValueError("a cache's tensors must be contiguous")
        self.index = _device_of(k, v, k_scale, v_scale)
        _int32("capacity", k.shape[2])
        self._tensors = (k, v, k_scale, v_scale)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    def c_struct(self):
        k, v, k_scale, v_scale = self._tensors
        return _Kv8Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.shape[2])

    @classmethod
    def empty(cls, B: int, kv_heads: int, capacity: int, d: int, device="cuda") -> "Kv8Cache":
        """A cache of zeros for ``capacity`` tokens (rounded up to whole blocks)."""
        import torch
        capacity = -(-capacity // KV8_BLOCK) * KV8_BLOCK
        codes = [torch.zeros(B, kv_heads, capacity, d, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                 for _ in range(2)]
        scales = [torch.ones(B, kv_heads, capacity // KV8_BLOCK, device=device) for _ in range(2)]
        return cls(*codes, *scales)

    @property
    def capacity(self) -> int:
        return int(self.k.shape[2])


@functools.lru_cache(maxsize=1024)
def _store_plan(cache_shape, k_shape, k_strides, v_shape, v_strides, k_dtype, v_dtype):
    B, kv_heads, _, d = cache_shape
    if len(k_shape) != 4:
        raise ValueError(f"expected [B, heads, L, d], got {tuple(k_shape)}")
    n = _int32("k", k_shape[2])
    strides = (_heads_strides("k", k_shape, k_strides, (B, kv_heads, k_shape[2], d)),
               _heads_strides("v", v_shape, v_strides, k_shape))
    code = _dtype_code(k_dtype, (NPA_DTYPE_BF16, NPA_DTYPE_FP16))
    if v_dtype != k_dtype:
        raise ValueError("k and v must have one dtype")
    return (code, B, kv_heads, d), n, strides


def kv8_store(cache: Kv8Cache, k, v, start: int = 0, starts=None, stream=None) -> None:
    """Writes bf16 or fp16 k, v [B, kv_heads, n, d] (strides as for
    ``cross_attention``) into the cache from token ``start`` on, or from
    ``starts[b]`` (int32 [B]) in batch row b."""
    _run_on(cache.index, stream, _kv8_store, cache, k, v, start, starts)


def _kv8_store(cache, k, v, start, starts, handle):
    import torch
    sizes, n, strides = _store_plan(cache.k.shape, k.shape, k.stride(), v.shape, v.stride(), k.dtype, v.dtype)
    if starts is not None and (starts.dtype != torch.int32 or starts.shape != sizes[1:2] or
                               not starts.is_contiguous()):
        raise ValueError(f"starts: expected a contiguous int32 tensor of {sizes[1]} positions")
    _device_of(cache.k, k, v, starts)
    code = lib().npa_kv8_store(k.data_ptr(), v.data_ptr(), cache.c_struct(), *sizes, _int32("start", start), _ptr(starts), n, *strides, handle)
    if code:
        raise NpaError(code, "npa_kv8_store")


@functools.lru_cache(maxsize=1024)
def _kv8_plan(index, split, q_shape, q_strides, cache_shape, Lk, q_dtype):
    B, kv_heads, capacity, d = cache_shape
    if len(q_shape) != 4:
        raise ValueError(f"expected [B, heads, L, d], got {tuple(q_shape)}")
    heads, Lq = (_int32("q", n) for n in q_shape[1:3])
    strides = _heads_strides("q", q_shape, q_strides, (B, heads, Lq, d))
    _dtype_code(q_dtype, (NPA_DTYPE_BF16,))
    Lk = capacity if Lk is None else _int32("n_tokens", Lk)
    nbytes = _planned_bytes(npa_cross_attention_workspace_size, B, heads, kv_heads, Lq, Lk, d) if split else 0   # on `index`
    return (B, heads, kv_heads, Lq, Lk, d), strides, _like_strides(q_shape, q_strides), nbytes


def kv8_cross_attention(q, cache: Kv8Cache, n_tokens: Optional[int] = None, kv_lens=None, key_mask=None,
                        scale: Optional[float] = None, out=None, split: bool = True, stream=None):
    """``cross_attention`` of bf16 q [B, heads, Lq, d] over the first
    ``n_tokens`` (default: all) tokens of an 8-bit cache."""
    return _run_on(cache.index, stream, _kv8_cross_attention, q, cache, n_tokens, kv_lens, key_mask, scale, out, split)


def _kv8_cross_attention(q, cache, n_tokens, kv_lens, key_mask, scale, out, split, handle):
    import torch
    n_tokens = None if n_tokens is None else operator.index(n_tokens)   # a tensor would be looked up by its identity
    sizes, q_strides, o_strides, nbytes = _kv8_plan(cache.index, bool(split), q.shape, q.stride(), cache.k.shape, n_tokens,
                                                    q.dtype)
    lens = mask = None
    if kv_lens is not None or key_mask is not None:
        _kept_keys(kv_lens, key_mask, sizes[0], sizes[4])
        lens, mask = _ptr(kv_lens), _ptr(key_mask)
    _device_of(cache.k, q, kv_lens, key_mask, out)
    if out is None:
        out = torch.empty_like(q)
    else:
        if out.dtype != q.dtype:
            raise ValueError("out must have q's dtype")
        o_strides = _heads_strides("out", out.shape, out.stride(), q.shape)
    ws = _empty_bytes(nbytes, q)
    code = lib().npa_kv8_cross_attention_fwd(
        q.data_ptr(), cache.c_struct(), out.data_ptr(), *sizes, q_strides, o_strides, lens, mask, _scale(scale),
        ws.data_ptr() if nbytes else None, nbytes, handle)
    if code:
        raise NpaError(code, "npa_kv8_cross_attention_fwd")
    return out


_ACTIVATIONS = {None: NPA_ACT_NONE, "none": NPA_ACT_NONE, "silu": NPA_ACT_SILU}


@functools.lru_cache(maxsize=1024)
def _norm_plan(index, groups, act, x_shape, x_strides, x_dtype, w_shape, w_strides, w_dtype, b_shape, b_strides, b_dtype):
    """((dtype codes and sizes), x's strides, activation, workspace bytes)."""
    if len(x_shape) != 3:
        raise ValueError(f"expected [B, N, C], got {tuple(x_shape)}")
    if act not in _ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}")
    B, N, C = (_int32("x", n) for n in x_shape)
    groups = _int32("groups", groups)
    code = wcode = _dtype_code(x_dtype, (NPA_DTYPE_BF16, NPA_DTYPE_FP16, NPA_DTYPE_FP32))
    for name, shape, strides, dtype in (("weight", w_shape, w_strides, w_dtype), ("bias", b_shape, b_strides, b_dtype)):
        if shape is None:
            continue
        if tuple(shape) != (C,) or (C > 1 and strides != (1,)):
            raise ValueError(f"{name}: expected a contiguous [{C}] tensor")
        wcode = _dtype_code(dtype, (code, NPA_DTYPE_FP32))
    if w_dtype is not None and b_dtype is not None and w_dtype != b_dtype:
        raise ValueError("weight and bias must have one dtype")
    if C > 1 and x_strides[2] != 1:
        raise ValueError("channels must be contiguous")
    nbytes = _planned_bytes(npa_group_norm_workspace_size, code, B, N, C, groups) if index >= 0 else 0   # on `index`
    return (code, wcode, B, N, C, groups), x_strides[:2], _ACTIVATIONS[act], nbytes


def group_norm(x, groups: int, weight=None, bias=None, eps: float = 1e-5, act: Optional[str] = None, out=None,
               stream=None):
    """Group norm with an activation (None or "silu") on a torch bf16, fp16 or
    fp32 CUDA tensor x [B, N, C], channels last and contiguous, batch and token
    strides free; weight and bias [C] of x's dtype or float32. ``out`` is laid
    out like x by default; ``out=x`` works in place. (A channels-last [B, C, H, W] tensor is ``x.permute(0, 2, 3,
    1).flatten(1, 2)``.)"""
    index = x.get_device()
    if index < 0:
        return _group_norm(index, x, groups, weight, bias, eps, act, out, 0)
    return _run_on(index, stream, _group_norm, index, x, groups, weight, bias, eps, act, out)


def _group_norm(index, x, groups, weight, bias, eps, act, out, handle):
    import torch
    w = (None, None, None) if weight is None else (weight.shape, weight.stride(), weight.dtype)
    b = (None, None, None) if bias is None else (bias.shape, bias.stride(), bias.dtype)
    sizes, xs, act_code, nbytes = _norm_plan(index, operator.index(groups), act, x.shape, x.stride(), x.dtype, *w, *b)
    _device_of(x, weight, bias, out)
    if out is None:
        out = torch.empty_like(x)
    elif out.dtype != x.dtype or out.shape != x.shape:
        raise ValueError("out must have x's shape and dtype")
    ys = out.stride()
    if ys[2] != 1 and x.shape[2] > 1:
        raise ValueError("channels must be contiguous")
    ws = _empty_bytes(nbytes, x)
    code = lib().npa_group_norm_act(x.data_ptr(), None if weight is None else weight.data_ptr(),
                                    None if bias is None else bias.data_ptr(), out.data_ptr(), *sizes, *xs, ys[0], ys[1],
                                    float(eps), act_code, ws.data_ptr() if nbytes else None, nbytes, handle)
    if code:
        raise NpaError(code, "npa_group_norm_act")
    return out
