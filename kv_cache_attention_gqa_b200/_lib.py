"""ctypes binding of the C ABI in ``include/gqa.h``: argument marshalling only.

Every step of the computation runs in the CUDA library ``libgqa_b200.so``; this module checks
tensor shapes and dtypes, allocates outputs with PyTorch (device memory is plumbing), passes raw
device pointers and the current CUDA stream, and turns status codes into exceptions.  There is no
fallback: if the library is missing, importing this module raises.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libgqa_b200.so")

GQA_OK = 0
STATUS_NAMES = {
    0: "GQA_OK",
    1: "GQA_ERR_INVALID_ARG",
    2: "GQA_ERR_UNSUPPORTED",
    3: "GQA_ERR_CUDA",
    4: "GQA_ERR_DEVICE",
    5: "GQA_ERR_WORKSPACE",
}
GQA_BF16, GQA_FP32 = 0, 1
DEVERR_NAMES = {0: "none", 1: "kv_len out of range", 2: "position out of range",
                3: "query with no visible key", 4: "pipeline wait timed out",
                5: "block-table entry out of range"}

# name -> (restype, argtypes), mirroring include/gqa.h
_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L3 = ctypes.POINTER(ctypes.c_int64)  # three strides (host memory)


class _ScoreMod(ctypes.Structure):
    """gqa_score_mod"""

    _fields_ = [("softcap", _F), ("alibi_slopes", _P), ("key_range", _P)]


_M = ctypes.POINTER(_ScoreMod)
SIGNATURES = {
    "gqa_prefill": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P]),
    "gqa_decode_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "gqa_decode": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I, _P, _Z, _I, _P]),
    "gqa_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P]),
    "kv_append": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "gqa_decode_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                              _I, _P, _Z, _I, _P]),
    "kv_append_paged": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "gqa_prefill_backward_workspace_size": (_Z, [_I, _I, _I]),
    "gqa_mla_decode_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "gqa_mla_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _Z, _I, _P]),
    "gqa_prefill_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                  _F, _I, _I, _I, _P, _Z, _P]),
    "gqa_rope": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _L3, _L3, _I, _I, _F, _I, _P]),
    "kv_rope_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _L3, _L3,
                            _L3, _I, _F, _I, _P]),
    "kv_rope_append_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _I,
                                  _I, _I, _L3, _L3, _L3, _I, _F, _I, _P]),
    "gqa_kv_weights_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "gqa_kv_weights": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _I, _P, _Z, _P]),
    "gqa_kv_weights_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _I,
                                  _P, _Z, _P]),
    "kv_evict": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "kv_evict_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "gqa_prefill_mod_workspace_size": (_Z, [_I, _I, _I, _I]),
    "gqa_prefill_mod": (_I, [_P, _P, _P, _P, _P, _P, _P, _M, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P, _Z, _P]),
    "gqa_prefill_backward_mod_workspace_size": (_Z, [_I, _I, _I, _I]),
    "gqa_prefill_backward_mod": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _M, _I, _I, _I, _I, _I, _I,
                                      _F, _I, _I, _I, _P, _Z, _P]),
    "gqa_decode_mod_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "gqa_decode_mod": (_I, [_P, _P, _P, _P, _P, _P, _P, _M, _I, _I, _I, _I, _I, _F, _I, _I, _P, _Z, _I, _P]),
    "gqa_decode_paged_mod": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _M, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                                  _I, _P, _Z, _I, _P]),
    "gqa_get_device_error": (_I, [ctypes.POINTER(_I), _P]),
    "gqa_status_string": (ctypes.c_char_p, [_I]),
    "gqa_version": (ctypes.c_char_p, []),
    "gqa_debug_expire_waits": (_I, [_I]),
}


class GQAError(RuntimeError):
    """A non-OK status returned by the library."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(or `python kv_cache_attention_gqa_b200/build.py`). There is no fallback implementation."
        )
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()


def _check(fn: str, status: int) -> None:
    if status != GQA_OK:
        raise GQAError(fn, status)


def version() -> str:
    return _lib.gqa_version().decode()


def status_string(status: int) -> str:
    return _lib.gqa_status_string(status).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GQA_BF16
    if t.dtype == torch.float32:
        return GQA_FP32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 (tensor-core path) or fp32 (check mode)")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    """Every tensor given is a contiguous CUDA tensor on the current device (the library launches on
    the current device and its current stream)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous (row-major)")
        if dev is None:
            dev = torch.cuda.current_device()
        if t.device.index != dev:
            raise ValueError(f"tensors must live on the current CUDA device (cuda:{dev}), not {t.device}")


def _int_vec(x, B: int, device, name: str):
    """Device int32[B] from None / int / sequence / tensor (None stays None = library default)."""
    if x is None:
        return None
    if (isinstance(x, torch.Tensor) and x.is_cuda and x.device == device and x.dtype == torch.int32 and x.is_contiguous()):
        if x.numel() != B:
            raise ValueError(f"{name} must have {B} entries")
        return x
    if isinstance(x, int):
        x = [x] * B
    t = torch.as_tensor(x, dtype=torch.int32, device=device).contiguous()
    if t.numel() != B:
        raise ValueError(f"{name} must have {B} entries")
    return t


def _out(out, shape, dtype, device):
    """The output tensor: a new one, or the caller's after checking its shape and dtype (the kernels
    write every element of ``shape``; a smaller buffer would be overrun)."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError(f"out must be {dtype} of shape {tuple(shape)}, not {out.dtype} {tuple(out.shape)}")
    return out


def _ws_bytes(ws) -> int:
    """Byte size of a caller workspace, which must be a contiguous tensor on the current device."""
    _need_cuda(ws)
    return ws.numel() * ws.element_size()


def _scale(scale) -> float:
    """None -> 0.0, which the C ABI reads as its default 1/sqrt(d_h) (MLA: 1/sqrt(d_qk))."""
    return 0.0 if scale is None else float(scale)


# The current device's index, without torch.cuda.current_device's check that CUDA is up: for calls that have seen a
# CUDA tensor.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# The raw handle of a device's current stream (torch.cuda.current_stream() builds an object around it, which costs more
# than the launch of a small kernel), and whether that stream is capturing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _stream():
    """The raw handle of the current device's current stream."""
    return _raw_stream(_device())


def debug_expire_waits(enable: bool) -> None:
    """Failure-detection test hook (gqa_debug_expire_waits): while enabled, bf16 prefill and
    contiguous bf16 decode make one bounded wait run out, so the call reports a timeout."""
    _check("gqa_debug_expire_waits", _lib.gqa_debug_expire_waits(1 if enable else 0))


def get_device_error() -> int:
    """Synchronise the current stream, read and clear the sticky device error word."""
    code = ctypes.c_int(0)
    torch.cuda.init()
    st = _lib.gqa_get_device_error(ctypes.byref(code), _stream())
    if st not in (GQA_OK, 4):
        raise GQAError("gqa_get_device_error", st)
    return code.value


def kv_append(k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
              v_new: torch.Tensor, pos) -> None:
    """cache[b, g, pos[b] + t] = new[b, g, t] for t < S_new (in place, bit-exact)."""
    _need_cuda(k_cache, v_cache, k_new, v_new)
    B, h_kv, T_max, d_h = k_cache.shape
    if v_cache.shape != k_cache.shape or k_new.shape != v_new.shape:
        raise ValueError("shape mismatch")
    if k_new.dim() != 4 or k_new.shape[0] != B or k_new.shape[1] != h_kv or k_new.shape[3] != d_h:
        raise ValueError("k_new must be (B, h_kv, S_new, d_h)")
    dt = _dtype_code(k_cache)
    if any(t.dtype != k_cache.dtype for t in (v_cache, k_new, v_new)):
        raise TypeError("all four tensors must share one dtype")
    pos_t = _int_vec(pos, B, k_cache.device, "pos")
    _check("kv_append", _lib.kv_append(_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                                       _ptr(pos_t), B, h_kv, k_new.shape[2], T_max, d_h, dt, _stream()))


def _score_mod(softcap: float, alibi_slopes, key_range, h_q: int, shape):
    """gqa_score_mod of a call's keyword arguments, or None when none is set."""
    if not softcap and alibi_slopes is None and key_range is None:
        return None
    _need_cuda(alibi_slopes, key_range)
    if alibi_slopes is not None and (alibi_slopes.dtype != torch.float32 or tuple(alibi_slopes.shape) != (h_q,)):
        raise ValueError(f"alibi_slopes must be float32 of shape ({h_q},)")
    if key_range is not None and (key_range.dtype != torch.int32 or tuple(key_range.shape) != shape):
        raise ValueError(f"key_range must be int32 of shape {shape}")
    return _ScoreMod(float(softcap), _ptr(alibi_slopes), _ptr(key_range))


def key_ranges(doc_ids: torch.Tensor, *, prefix_len=None, causal: bool = True) -> torch.Tensor:
    """``key_range`` (B, S, 2) int32 for documents packed into the S cached rows of each sequence: neighbours with equal
    ``doc_ids`` (B, S) are one document, a negative id is padding (its rows see nothing). Rows see the keys of their
    document at and before them (``causal``), or all of them; ``prefix_len`` (an int, or ids' shape: the length for
    each row's document): the first rows of a document are seen by all of it. Use with ``causal=False``."""
    B, S = doc_ids.shape
    at = torch.arange(S, device=doc_ids.device).expand(B, S)
    new = torch.ones_like(doc_ids, dtype=torch.bool)
    new[:, 1:] = doc_ids[:, 1:] != doc_ids[:, :-1]
    lo = torch.where(new, at, 0).cummax(1).values
    last = torch.ones_like(new)
    last[:, :-1] = new[:, 1:]
    hi = torch.where(last, at + 1, S).flip(1).cummin(1).values.flip(1)
    if causal:
        end = at + 1
        if prefix_len is not None:
            end = torch.maximum(end, torch.minimum(lo + prefix_len, hi))
        hi = end
    pad = doc_ids < 0
    return torch.stack([lo.masked_fill(pad, 0), hi.masked_fill(pad, 0)], -1).to(torch.int32)


def prefill(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *, q_start=None,
            kv_len=None, scale: float | None = None, causal: bool = True, window: int = 0,
            softcap: float = 0.0, alibi_slopes=None, key_range=None, out=None, return_lse: bool = False):
    """Grouped-query attention of q (B, h_q, S_q, d_h) over the cache (B, h_kv, T_max, d_h).
    ``window`` > 0: sliding window, row at position p sees keys p - window < j <= p. ``softcap`` > 0: scores s become
    softcap tanh(s / softcap); ``alibi_slopes`` (h_q,) fp32: slope |p - j| is subtracted; ``key_range`` (B, S_q, 2)
    int32: a row sees only keys lo <= j < hi (see ``key_ranges``)."""
    _need_cuda(q, k_cache, v_cache, out)
    B, h_q, S_q, d_h = q.shape
    Bk, h_kv, T_max, dk = k_cache.shape
    if (Bk, dk) != (B, d_h) or v_cache.shape != k_cache.shape:
        raise ValueError("q / k_cache / v_cache shapes disagree")
    dt = _dtype_code(q)
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    out = torch.empty_like(q) if out is None else _out(out, q.shape, q.dtype, q.device)
    lse = q.new_empty((B, h_q, S_q), dtype=torch.float32) if return_lse else None
    qs = _int_vec(q_start, B, q.device, "q_start")
    kl = _int_vec(kv_len, B, q.device, "kv_len")
    scale = _scale(scale)
    mod = _score_mod(softcap, alibi_slopes, key_range, h_q, (B, S_q, 2))
    if mod is not None:
        # the ranges' hulls: scratch of this call (a capture keeps it in its own pool)
        need = _lib.gqa_prefill_mod_workspace_size(B, h_q, h_kv, S_q) if key_range is not None else 0
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        _check("gqa_prefill_mod", _lib.gqa_prefill_mod(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(qs), _ptr(kl), mod, B, h_q, h_kv, S_q,
            T_max, d_h, scale, 1 if causal else 0, int(window), dt, _ptr(ws), need, _stream()))
        return (out, lse) if return_lse else out
    _check("gqa_prefill", _lib.gqa_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse),
                                           _ptr(qs), _ptr(kl), B, h_q, h_kv, S_q, T_max, d_h, scale,
                                           1 if causal else 0, int(window), dt, _stream()))
    return (out, lse) if return_lse else out


def decode_workspace_size(B: int, h_q: int, h_kv: int, T_max: int, d_h: int, dtype=torch.bfloat16,
                          num_splits: int = 0, modified: bool = False) -> int:
    """Bytes of workspace of a decode call (``modified``: with softcap, alibi_slopes or key_range)."""
    dt = GQA_BF16 if dtype == torch.bfloat16 else GQA_FP32
    name = "gqa_decode_mod_workspace_size" if modified else "gqa_decode_workspace_size"
    n = getattr(_lib, name)(B, h_q, h_kv, T_max, d_h, dt, num_splits)
    if n == 0:
        raise GQAError(name, 1)
    return n


_HEADER = 256  # bytes of a decode workspace that have to start at zero (the ticket counter's)


def _decode_workspace(ws, need: int, device):
    """A decode's workspace and its size: the caller's, or the stream's cached one. A captured call takes one from the
    capture's own pool and clears its counters in the graph (1 us; a caller's ``ws`` saves it), so that graphs captured
    on one stream can run at once, in any order, and a cached workspace that grows later takes nothing from them."""
    if ws is not None:
        return ws, _ws_bytes(ws)
    if _capturing():
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        ws[:_HEADER].zero_()
    else:
        ws = workspace(need, device)
    return ws, ws.numel()


_ws_lock = threading.Lock()
_ws_cache: dict = {}
_ws_sizes: dict = {}


def workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled, 256-byte aligned device workspace of at least ``nbytes``, cached per device
    and stream (every completed decode leaves its counter region at zero again)."""
    dev = torch.device(device)
    index = torch.cuda.current_device() if dev.index is None else dev.index
    key = (index, _raw_stream(index))
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
            _ws_cache[key] = buf
    return buf


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *, kv_len=None,
           q_pos=None, scale: float | None = None, window: int = 0, num_splits: int = 0,
           softcap: float = 0.0, alibi_slopes=None, key_range=None, out=None,
           return_lse: bool = False, ws: torch.Tensor | None = None):
    """Split-KV decode of q (B, h_q, d_h) over the cache (B, h_kv, T_max, d_h).
    ``window`` > 0: sliding window, the query at q_pos sees keys q_pos - window < j <= q_pos.
    ``softcap``, ``alibi_slopes``: as in ``prefill``; ``key_range`` (B, 2): the keys each sequence sees."""
    _need_cuda(q, k_cache, v_cache, out)
    B, h_q, d_h = q.shape
    Bk, h_kv, T_max, dk = k_cache.shape
    if (Bk, dk) != (B, d_h) or v_cache.shape != k_cache.shape:
        raise ValueError("q / k_cache / v_cache shapes disagree")
    dt = _dtype_code(q)
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    out = torch.empty_like(q) if out is None else _out(out, q.shape, q.dtype, q.device)
    lse = q.new_empty((B, h_q), dtype=torch.float32) if return_lse else None
    kl = _int_vec(kv_len, B, q.device, "kv_len")
    qp = _int_vec(q_pos, B, q.device, "q_pos")
    scale = _scale(scale)
    mod = _score_mod(softcap, alibi_slopes, key_range, h_q, (B, 2))
    key = (B, h_q, h_kv, T_max, d_h, dt, num_splits, q.device.index, mod is None)
    need = _ws_sizes.get(key)
    if need is None:
        need = _ws_sizes[key] = decode_workspace_size(B, h_q, h_kv, T_max, d_h, q.dtype, num_splits, mod is not None)
    ws, nws = _decode_workspace(ws, need, q.device)
    if mod is not None:
        _check("gqa_decode_mod", _lib.gqa_decode_mod(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(kl), _ptr(qp), mod, B, h_q, h_kv, T_max,
            d_h, scale, int(window), dt, _ptr(ws), nws, num_splits, _stream()))
        return (out, lse) if return_lse else out
    _check("gqa_decode", _lib.gqa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse),
                                         _ptr(kl), _ptr(qp), B, h_q, h_kv, T_max, d_h, scale,
                                         int(window), dt, _ptr(ws), nws, num_splits, _stream()))
    return (out, lse) if return_lse else out


def decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *, kv_len=None,
                   q_pos=None, scale: float | None = None, window: int = 0, num_splits: int = 0,
                   out=None, return_lse: bool = False):
    """gqa_decode_noalloc: the decode with the library's fixed device scratch array instead of a
    caller workspace, for callers that cannot allocate device memory (the output buffer may be
    passed in as ``out``). Overlapping calls on different streams race on that array."""
    _need_cuda(q, k_cache, v_cache, out)
    B, h_q, d_h = q.shape
    Bk, h_kv, T_max, dk = k_cache.shape
    if (Bk, dk) != (B, d_h) or v_cache.shape != k_cache.shape:
        raise ValueError("q / k_cache / v_cache shapes disagree")
    dt = _dtype_code(q)
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    out = torch.empty_like(q) if out is None else _out(out, q.shape, q.dtype, q.device)
    lse = q.new_empty((B, h_q), dtype=torch.float32) if return_lse else None
    kl = _int_vec(kv_len, B, q.device, "kv_len")
    qp = _int_vec(q_pos, B, q.device, "q_pos")
    scale = _scale(scale)
    _check("gqa_decode_noalloc", _lib.gqa_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                                         _ptr(lse), _ptr(kl), _ptr(qp), B, h_q, h_kv, T_max,
                                                         d_h, scale, int(window), dt, num_splits, _stream()))
    return (out, lse) if return_lse else out


def _block_table(block_table, B: int, device) -> torch.Tensor:
    t = block_table
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == torch.device(device)
            and t.dtype == torch.int32 and t.is_contiguous()):
        t = torch.as_tensor(block_table, dtype=torch.int32, device=device).contiguous()
    if t.dim() != 2 or t.shape[0] != B:
        raise ValueError("block_table must be (B, max_pages)")
    return t


def _pool_shape(k_pages: torch.Tensor, v_pages: torch.Tensor):
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages / v_pages must both be (num_pages, h_kv, page_size, d_h)")
    return k_pages.shape


def decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table, *,
                 kv_len=None, q_pos=None, scale: float | None = None, window: int = 0,
                 num_splits: int = 0, softcap: float = 0.0, alibi_slopes=None, key_range=None, out=None,
                 return_lse: bool = False, ws: torch.Tensor | None = None):
    """Split-KV decode of q (B, h_q, d_h) over a paged cache: pools (num_pages, h_kv, page_size,
    d_h) and block_table (B, max_pages) int32; position t of sequence b is row t % page_size of
    page block_table[b, t // page_size]. Modified scores as in ``decode``."""
    _need_cuda(q, k_pages, v_pages, out)
    B, h_q, d_h = q.shape
    num_pages, h_kv, page_size, dk = _pool_shape(k_pages, v_pages)
    if dk != d_h:
        raise ValueError("q and the page pools disagree on d_h")
    dt = _dtype_code(q)
    if k_pages.dtype != q.dtype or v_pages.dtype != q.dtype:
        raise TypeError("q, k_pages and v_pages must share one dtype")
    bt = _block_table(block_table, B, q.device)
    max_pages = bt.shape[1]
    out = torch.empty_like(q) if out is None else _out(out, q.shape, q.dtype, q.device)
    lse = q.new_empty((B, h_q), dtype=torch.float32) if return_lse else None
    kl = _int_vec(kv_len, B, q.device, "kv_len")
    qp = _int_vec(q_pos, B, q.device, "q_pos")
    scale = _scale(scale)
    T_max = max_pages * page_size
    mod = _score_mod(softcap, alibi_slopes, key_range, h_q, (B, 2))
    key = (B, h_q, h_kv, T_max, d_h, dt, num_splits, q.device.index, mod is None)
    need = _ws_sizes.get(key)
    if need is None:
        need = _ws_sizes[key] = decode_workspace_size(B, h_q, h_kv, T_max, d_h, q.dtype, num_splits, mod is not None)
    ws, nws = _decode_workspace(ws, need, q.device)
    if mod is not None:
        _check("gqa_decode_paged_mod", _lib.gqa_decode_paged_mod(
            _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(out), _ptr(lse), _ptr(kl), _ptr(qp), _ptr(bt), mod, B, h_q,
            h_kv, num_pages, page_size, max_pages, d_h, scale, int(window), dt, _ptr(ws), nws, num_splits, _stream()))
        return (out, lse) if return_lse else out
    _check("gqa_decode_paged", _lib.gqa_decode_paged(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(out), _ptr(lse), _ptr(kl), _ptr(qp), _ptr(bt),
        B, h_q, h_kv, num_pages, page_size, max_pages, d_h, scale, int(window), dt, _ptr(ws), nws, num_splits,
        _stream()))
    return (out, lse) if return_lse else out


def kv_append_paged(k_pages: torch.Tensor, v_pages: torch.Tensor, k_new: torch.Tensor,
                    v_new: torch.Tensor, pos, block_table) -> None:
    """Write new[b, g, t] at logical position pos[b] + t of a paged cache (in place, bit-exact)."""
    _need_cuda(k_pages, v_pages, k_new, v_new)
    num_pages, h_kv, page_size, d_h = _pool_shape(k_pages, v_pages)
    if k_new.dim() != 4 or k_new.shape != v_new.shape or k_new.shape[1] != h_kv or k_new.shape[3] != d_h:
        raise ValueError("k_new / v_new must be (B, h_kv, S_new, d_h)")
    B = k_new.shape[0]
    dt = _dtype_code(k_pages)
    if any(t.dtype != k_pages.dtype for t in (v_pages, k_new, v_new)):
        raise TypeError("all four tensors must share one dtype")
    bt = _block_table(block_table, B, k_pages.device)
    pos_t = _int_vec(pos, B, k_pages.device, "pos")
    _check("kv_append_paged", _lib.kv_append_paged(
        _ptr(k_pages), _ptr(v_pages), _ptr(k_new), _ptr(v_new), _ptr(pos_t), _ptr(bt), B, h_kv,
        k_new.shape[2], num_pages, page_size, bt.shape[1], d_h, dt, _stream()))


def prefill_backward(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, o: torch.Tensor,
                     d_o: torch.Tensor, lse: torch.Tensor, *, q_start=None, kv_len=None,
                     scale: float | None = None, causal: bool = True, window: int = 0,
                     softcap: float = 0.0, alibi_slopes=None, key_range=None,
                     ws: torch.Tensor | None = None):
    """Gradients (dq, dk, dv) of ``prefill`` for the upstream gradient ``d_o``; ``o`` and ``lse``
    are the forward's outputs (``prefill(..., return_lse=True)``, the same arguments). dk, dv have the cache's
    shape, zero past each kv_len. ``alibi_slopes`` are constants."""
    _need_cuda(q, k_cache, v_cache, o, d_o, lse)
    B, h_q, S_q, d_h = q.shape
    Bk, h_kv, T_max, dk_ = k_cache.shape
    if (Bk, dk_) != (B, d_h) or v_cache.shape != k_cache.shape or o.shape != q.shape or d_o.shape != q.shape:
        raise ValueError("q / k_cache / v_cache / o / d_o shapes disagree")
    if lse.shape != (B, h_q, S_q) or lse.dtype != torch.float32:
        raise ValueError("lse must be fp32 (B, h_q, S_q)")
    dt = _dtype_code(q)
    if any(t.dtype != q.dtype for t in (k_cache, v_cache, o, d_o)):
        raise TypeError("q, k_cache, v_cache, o and d_o must share one dtype")
    dq = torch.empty_like(q)
    dk = torch.empty_like(k_cache)
    dv = torch.empty_like(v_cache)
    qs = _int_vec(q_start, B, q.device, "q_start")
    kl = _int_vec(kv_len, B, q.device, "kv_len")
    scale = _scale(scale)
    mod = _score_mod(softcap, alibi_slopes, key_range, h_q, (B, S_q, 2))
    need = (_lib.gqa_prefill_backward_workspace_size(B, h_q, S_q) if mod is None
            else _lib.gqa_prefill_backward_mod_workspace_size(B, h_q, h_kv, S_q))
    if ws is None or _ws_bytes(ws) < need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    if mod is not None:
        _check("gqa_prefill_backward_mod", _lib.gqa_prefill_backward_mod(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(d_o), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(qs),
            _ptr(kl), mod, B, h_q, h_kv, S_q, T_max, d_h, scale, 1 if causal else 0, int(window), dt, _ptr(ws),
            _ws_bytes(ws), _stream()))
        return dq, dk, dv
    _check("gqa_prefill_backward", _lib.gqa_prefill_backward(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(d_o), _ptr(lse), _ptr(dq), _ptr(dk),
        _ptr(dv), _ptr(qs), _ptr(kl), B, h_q, h_kv, S_q, T_max, d_h, scale, 1 if causal else 0,
        int(window), dt, _ptr(ws), _ws_bytes(ws), _stream()))
    return dq, dk, dv


def mla_decode(q: torch.Tensor, cache: torch.Tensor, d_v: int = 512, *, kv_len=None, q_pos=None,
               scale: float | None = None, num_splits: int = 0, out=None, return_lse: bool = False,
               ws: torch.Tensor | None = None):
    """MLA decode over a latent cache: q (B, h_q, d_qk) = [absorbed latent query | rotary part],
    cache (B, T_max, d_qk) = [latent | rotary key]; returns the latent output (B, h_q, d_v) (the
    value rows are cache[..., :d_v]). ``scale`` should be the model's softmax scale."""
    _need_cuda(q, cache, out)
    B, h_q, d_qk = q.shape
    Bc, T_max, dc = cache.shape
    if (Bc, dc) != (B, d_qk):
        raise ValueError("q and cache shapes disagree")
    dt = _dtype_code(q)
    if cache.dtype != q.dtype:
        raise TypeError("q and cache must share one dtype")
    out = _out(out, (B, h_q, d_v), q.dtype, q.device)
    lse = torch.empty((B, h_q), dtype=torch.float32, device=q.device) if return_lse else None
    kl = _int_vec(kv_len, B, q.device, "kv_len")
    qp = _int_vec(q_pos, B, q.device, "q_pos")
    scale = _scale(scale)
    key = ("mla", B, h_q, T_max, d_v, dt, num_splits, q.device.index)
    need = _ws_sizes.get(key)
    if need is None:
        need = _lib.gqa_mla_decode_workspace_size(B, h_q, T_max, d_v, dt, num_splits)
        if need == 0:
            raise GQAError("gqa_mla_decode_workspace_size", 1)
        _ws_sizes[key] = need
    ws, nws = _decode_workspace(ws, need, q.device)
    _check("gqa_mla_decode", _lib.gqa_mla_decode(
        _ptr(q), _ptr(cache), _ptr(out), _ptr(lse), _ptr(kl), _ptr(qp), B, h_q, T_max, d_qk, d_v,
        scale, dt, _ptr(ws), nws, num_splits, _stream()))
    return (out, lse) if return_lse else out


def _on_device(*ts):
    """Every tensor given is a CUDA tensor on the current device (as _need_cuda, for strided inputs)."""
    dev = _device() if ts[0].is_cuda else -2
    for t in ts:
        if t is None or t.get_device() == dev:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        raise ValueError(f"tensors must live on the current CUDA device (cuda:{dev}), not {t.device}")


def _rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """A (B, heads, S, d) tensor whose rows have adjacent elements; the other strides are free."""
    if t.dim() != 4:
        raise ValueError(f"{name} must have the dimensions (B, heads, S, d)")
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent (last stride 1)")
    return t


@functools.lru_cache(maxsize=1024)
def _stride_array(strides):
    return (ctypes.c_int64 * 3)(*strides[:3])


def _strides(t: torch.Tensor):
    """Host int64[3] of t's strides (read-only; one array per distinct strides)."""
    return _stride_array(t.stride())


def _positions(positions, B: int, S: int, device, name: str):
    """(device int32 tensor, 1 when it holds a position per token): (B, S) per token, else first positions (B)."""
    if isinstance(positions, torch.Tensor) and positions.dim() == 2:
        if tuple(positions.shape) != (B, S):
            raise ValueError(f"{name} must be ({B},) first positions or ({B}, {S}) positions")
        return positions.to(device=device, dtype=torch.int32).contiguous(), 1
    return _int_vec(positions, B, device, name), 0


def _inv_freq(inv_freq: torch.Tensor, d: int, offset: int) -> torch.Tensor:
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise TypeError("inv_freq must be a 1-D float64 tensor (see rope_frequencies)")
    if not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous")
    if inv_freq.numel() < 1 or offset < 0 or offset + 2 * inv_freq.numel() > d:
        raise ValueError(f"the rotated segment [{offset}, {offset + 2 * inv_freq.numel()}) must lie in a row of {d}")
    return inv_freq


def rope_frequencies(d_rot: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     ramp: str = "turns", device="cuda"):
    """Angles per position of the d_rot / 2 pairs and the magnitude for ``rope``: (inv_freq float64
    tensor, scale). Without scaling inv_freq[i] = base ** (-2 i / d_rot) and scale = 1. For contexts
    ``factor`` times longer than ``original_length``:
    ``linear`` divides every frequency by factor; ``ntk`` raises the base so that the slowest pair is
    slowed by factor and the fastest is kept; ``yarn`` keeps pairs that turn at least beta_fast times over
    the original length, divides those that turn at most beta_slow times, blends in between, and returns
    scale = 0.1 ln(factor) + 1. The blend is linear in the pair's turns (``ramp`` "turns", the method as published) or
    in its index ("index": from the last index with at least beta_fast turns to the first with at most beta_slow, within
    0 .. d_rot - 1; the usual code of models that ship with it). The pairs in between get other angles: take the one
    that the model was trained with."""
    if d_rot <= 0 or d_rot % 2:
        raise ValueError("d_rot must be even and positive")
    if not (base > 0 and factor >= 1.0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(d_rot // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk" and d_rot > 2:
        base = base * factor ** (d_rot / (d_rot - 2))
    f = base ** (-2.0 * i / d_rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_length <= 0 or not beta_fast > beta_slow:
            raise ValueError("yarn needs original_length > 0 and beta_fast > beta_slow")
        if ramp == "turns":
            turns = original_length * f / (2.0 * math.pi)
            keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        elif ramp == "index":
            if not (base > 1.0 and beta_slow > 0.0):
                raise ValueError("a ramp over the index needs base > 1 and beta_slow > 0")
            # the index at which original_length base ** (-2 i / d_rot) / (2 pi) turns are beta
            at = [d_rot * math.log(original_length / (2.0 * math.pi * b)) / (2.0 * math.log(base)) for b in (beta_fast, beta_slow)]
            first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d_rot - 1)
            keep = 1.0 - ((i - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
        else:
            raise ValueError(f"unknown ramp {ramp!r}: 'turns' or 'index'")
        f = f * (keep + (1.0 - keep) / factor)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}: None, 'linear', 'ntk' or 'yarn'")
    return f.to(device), scale


def rope(x: torch.Tensor, inv_freq: torch.Tensor, positions, *, offset: int = 0, interleaved: bool = False,
         inverse: bool = False, scale: float = 1.0, out=None) -> torch.Tensor:
    """Rotary positions of the rows x (B, h, S, d), any strides but the last: pair i of the
    2 * len(inv_freq) elements from ``offset`` on turns by position * inv_freq[i] and is multiplied by
    ``scale``; the other elements are copied. ``positions``: (B,) first positions or (B, S). Pairs are
    elements i and i + len(inv_freq) of the segment, or neighbours (``interleaved``). ``inverse`` turns
    back: it maps the gradient of the result to the gradient of x. Returns a contiguous tensor, or ``out``
    (which may be x itself)."""
    _on_device(x, inv_freq, out)
    _rows(x, "x")
    B, h, S, d = x.shape
    dt = _dtype_code(x)
    inv_freq = _inv_freq(inv_freq, d, offset)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _rows(_out(out, x.shape, x.dtype, x.device), "out")
        if any(n > 1 and st == 0 for n, st in zip(out.shape, out.stride())):
            raise ValueError("out must not be a broadcast tensor")
        if out.data_ptr() == x.data_ptr() and out.stride() != x.stride():
            raise ValueError("in place, out must have the strides of x")
    pos_t, per_token = _positions(positions, B, S, x.device, "positions")
    _check("gqa_rope", _lib.gqa_rope(
        _ptr(x), _ptr(out), _ptr(inv_freq), _ptr(pos_t), per_token, B, h, S, d, 2 * inv_freq.numel(), offset,
        _strides(x), _strides(out), 1 if interleaved else 0, 1 if inverse else 0, scale, dt, _stream()))
    return out


def _rope_append(q, k_new, v_new, k_cache, v_cache, h_kv, d, pos, inv_freq, positions, offset, q_out):
    """Checks and arguments shared by kv_rope_append and kv_rope_append_paged."""
    _on_device(q, k_new, v_new, inv_freq, k_cache, v_cache, q_out)
    _rows(q, "q"), _rows(k_new, "k_new"), _rows(v_new, "v_new")
    B, h_q, S, dq = q.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("the K and V caches must have one shape")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous (row-major)")
    new = (B, h_kv, S, d)
    if dq != d or k_new.shape != new or v_new.shape != new:
        raise ValueError("q must be (B, h_q, S, d) and k_new, v_new (B, h_kv, S, d)")
    dtype = q.dtype
    if k_new.dtype != dtype or v_new.dtype != dtype or k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError("q, k_new, v_new and the caches must share one dtype")
    dt = _dtype_code(q)
    inv_freq = _inv_freq(inv_freq, d, offset)
    pos_t = _int_vec(pos, B, q.device, "pos")
    if pos_t is None:
        raise ValueError("pos must be given")
    at, per_token = (None, 0) if positions is None else _positions(positions, B, S, q.device, "positions")
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _out(q_out, (B, h_q, S, d), dtype, q.device)
        if not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous (row-major)")
        if q_out.data_ptr() == q.data_ptr() and not q.is_contiguous():
            raise ValueError("in place, q must be contiguous")
    return B, h_q, S, dt, inv_freq, pos_t, at, per_token, q_out


def kv_rope_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, pos, inv_freq: torch.Tensor, *, positions=None, offset: int = 0,
                   interleaved: bool = False, scale: float = 1.0, q_out=None) -> torch.Tensor:
    """``rope`` of a step's q (B, h_q, S, d) and k_new (B, h_kv, S, d), with ``kv_append`` of the rotated
    k and of v_new at cache rows pos[b] + t (in place), in one launch; returns the rotated q (contiguous).
    ``positions``: as in ``rope``; None: a token's position is its cache row."""
    if k_cache.dim() != 4 or k_cache.shape[0] != q.shape[0]:
        raise ValueError("the caches must be (B, h_kv, T_max, d)")
    _, h_kv, T_max, d = k_cache.shape
    B, h_q, S, dt, inv_freq, pos_t, at, per_token, q_out = _rope_append(
        q, k_new, v_new, k_cache, v_cache, h_kv, d, pos, inv_freq, positions, offset, q_out)
    _check("kv_rope_append", _lib.kv_rope_append(
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        inv_freq.data_ptr(), pos_t.data_ptr(), _ptr(at), per_token, B, h_q, h_kv, S, T_max, d, 2 * inv_freq.numel(), offset, _strides(q),
        _strides(k_new), _strides(v_new), 1 if interleaved else 0, scale, dt, _stream()))
    return q_out


def kv_rope_append_paged(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor,
                         v_pages: torch.Tensor, pos, block_table, inv_freq: torch.Tensor, *, positions=None,
                         offset: int = 0, interleaved: bool = False, scale: float = 1.0,
                         q_out=None) -> torch.Tensor:
    """``kv_rope_append`` into a paged cache (pools and block table as in ``kv_append_paged``)."""
    num_pages, h_kv, page_size, d = _pool_shape(k_pages, v_pages)
    B, h_q, S, dt, inv_freq, pos_t, at, per_token, q_out = _rope_append(
        q, k_new, v_new, k_pages, v_pages, h_kv, d, pos, inv_freq, positions, offset, q_out)
    bt = _block_table(block_table, B, q.device)
    _check("kv_rope_append_paged", _lib.kv_rope_append_paged(
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), q_out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        inv_freq.data_ptr(), pos_t.data_ptr(), _ptr(at), per_token, bt.data_ptr(), B, h_q, h_kv, S, num_pages, page_size, bt.shape[1], d, 2 * inv_freq.numel(),
        offset, _strides(q), _strides(k_new), _strides(v_new), 1 if interleaved else 0, scale, dt, _stream()))
    return q_out


def _weights_args(q, k, lse, h_kv, T_max, d, weights, kv_len, q_start, ws):
    """Checks and arguments shared by kv_weights and kv_weights_paged. q and lse may lack the row dimension
    (one decoded token)."""
    _need_cuda(q, k, lse, weights)
    if q.dim() not in (3, 4) or lse.shape != q.shape[:-1] or q.shape[-1] != d:
        raise ValueError("q must be (B, h_q, S_q, d_h) or (B, h_q, d_h), and lse its rows")
    B, h_q = q.shape[:2]
    S = q.shape[2] if q.dim() == 4 else 1
    dt = _dtype_code(q)
    if k.dtype != q.dtype:
        raise TypeError("q and the cache must share one dtype")
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    accumulate = weights is not None
    weights = _out(weights, (B, h_kv, T_max), torch.float32, q.device)
    kl = _int_vec(kv_len, B, q.device, "kv_len")
    qs = _int_vec(q_start, B, q.device, "q_start")
    key = ("weights", B, h_q, h_kv, S, T_max, dt, q.get_device())
    need = _ws_sizes.get(key)
    if need is None:
        need = _ws_sizes[key] = _lib.gqa_kv_weights_workspace_size(B, h_q, h_kv, S, T_max, dt)
    if ws is None and need:
        # not the cached workspace: that one's zeroed header belongs to the decode calls
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    return B, h_q, S, dt, int(accumulate), weights, kl, qs, ws, 0 if ws is None else _ws_bytes(ws)


def kv_weights(q: torch.Tensor, k_cache: torch.Tensor, lse: torch.Tensor, *, q_start=None, kv_len=None,
               scale: float | None = None, causal: bool = True, window: int = 0, weights=None,
               ws: torch.Tensor | None = None) -> torch.Tensor:
    """Attention weight of every cached key, fp32 (B, h_kv, T_max): the sum over the group's heads and the
    query rows that see it of exp(scale q.k - lse). q (B, h_q, S_q, d_h) with lse (B, h_q, S_q) as returned
    by ``prefill``, or (B, h_q, d_h) with (B, h_q) by ``decode``. ``q_start`` None: the queries are the
    last S_q cached rows (``prefill``'s None is row 0: give both the same). ``weights`` given: the sums are added to its entries j < kv_len, in place. The scores
    are plain ones, so ``lse`` is one of a call without softcap, alibi_slopes and key_range."""
    if k_cache.dim() != 4 or k_cache.shape[0] != q.shape[0]:
        raise ValueError("k_cache must be (B, h_kv, T_max, d_h)")
    _, h_kv, T_max, d = k_cache.shape
    B, h_q, S, dt, acc, weights, kl, qs, ws, nws = _weights_args(q, k_cache, lse, h_kv, T_max, d, weights, kv_len,
                                                                 q_start, ws)
    _check("gqa_kv_weights", _lib.gqa_kv_weights(
        _ptr(q), _ptr(k_cache), _ptr(lse), _ptr(weights), _ptr(qs), _ptr(kl), B, h_q, h_kv, S, T_max, d,
        _scale(scale), 1 if causal else 0, int(window), acc, dt, _ptr(ws), nws, _stream()))
    return weights


def kv_weights_paged(q: torch.Tensor, k_pages: torch.Tensor, block_table, lse: torch.Tensor, *, q_start=None,
                     kv_len=None, scale: float | None = None, causal: bool = True, window: int = 0,
                     weights=None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """``kv_weights`` over a paged cache (pool and block table as in ``decode_paged``); weights are
    (B, h_kv, max_pages * page_size), by logical position."""
    num_pages, h_kv, page_size, d = _pool_shape(k_pages, k_pages)
    bt = _block_table(block_table, q.shape[0], q.device)
    max_pages = bt.shape[1]
    B, h_q, S, dt, acc, weights, kl, qs, ws, nws = _weights_args(q, k_pages, lse, h_kv, max_pages * page_size, d,
                                                                 weights, kv_len, q_start, ws)
    _check("gqa_kv_weights_paged", _lib.gqa_kv_weights_paged(
        _ptr(q), _ptr(k_pages), _ptr(lse), _ptr(weights), _ptr(qs), _ptr(kl), _ptr(bt), B, h_q, h_kv, S, num_pages,
        page_size, max_pages, d, _scale(scale), 1 if causal else 0, int(window), acc, dt, _ptr(ws), nws, _stream()))
    return weights


def _evict_args(k, v, weights, B, h_kv, T_max, T_out, budget, kv_len, weights_out, kept):
    """Checks and arguments shared by kv_evict and kv_evict_paged."""
    _need_cuda(k, v, weights, weights_out, kept)
    dt = _dtype_code(k)
    if v.dtype != k.dtype:
        raise TypeError("the caches must share one dtype")
    if weights.dtype != torch.float32 or tuple(weights.shape) != (B, h_kv, T_max):
        raise ValueError(f"weights must be float32 of shape {(B, h_kv, T_max)}")
    budget = int(budget)
    if budget < 1 or budget > T_out:
        raise ValueError(f"budget must be between 1 and {T_out}")
    if weights_out is None:
        if T_out != T_max:
            raise ValueError("weights_out must be given when the caches are not shortened in place")
        weights_out = weights
    _out(weights_out, (B, h_kv, T_out), torch.float32, weights.device)
    if kept is None:
        kept = weights.new_empty((B, h_kv, budget), dtype=torch.int32)
    else:
        _out(kept, (B, h_kv, budget), torch.int32, weights.device)
    new_len = weights.new_empty(B, dtype=torch.int32)
    return dt, budget, weights_out, kept, new_len, _int_vec(kv_len, B, weights.device, "kv_len")


def kv_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, budget: int, *, kv_len=None,
             sink: int = 0, recent: int = 0, k_out=None, v_out=None, weights_out=None, kept=None):
    """Shorten every KV head's rows to at most ``budget``: the first ``sink``, the last ``recent`` and the
    heaviest of the others (``weights`` from ``kv_weights``; ties to the lower row) move to the front in
    their order. In place, or into ``k_out``, ``v_out``, ``weights_out`` of (B, h_kv, T_out, d_h) and
    (B, h_kv, T_out). Weights past the new length become zero. Returns (kept, new_len): the rows kept
    (B, h_kv, budget) int32, -1 past the new length, and the new lengths (B,) int32. Keys keep their rotation; in the
    calls after it ``window``, ``alibi_slopes`` and ``key_range`` count the rows that are left."""
    _need_cuda(k_cache, v_cache, k_out, v_out)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache / v_cache must both be (B, h_kv, T_max, d_h)")
    B, h_kv, T_max, d = k_cache.shape
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out must be given together")
    T_out = T_max
    if k_out is None:
        k_out, v_out = k_cache, v_cache
    else:
        if k_out.dim() != 4 or v_out.shape != k_out.shape or tuple(k_out.shape) != (B, h_kv, k_out.shape[2], d):
            raise ValueError("k_out / v_out must both be (B, h_kv, T_out, d_h)")
        if k_out.dtype != k_cache.dtype or v_out.dtype != k_cache.dtype:
            raise TypeError("the caches must share one dtype")
        if weights_out is None:
            raise ValueError("weights_out must be given with k_out and v_out")
        T_out = k_out.shape[2]
    dt, budget, weights_out, kept, new_len, kl = _evict_args(k_cache, v_cache, weights, B, h_kv, T_max, T_out,
                                                             budget, kv_len, weights_out, kept)
    _check("kv_evict", _lib.kv_evict(
        _ptr(k_cache), _ptr(v_cache), _ptr(k_out), _ptr(v_out), _ptr(weights), _ptr(weights_out), _ptr(kept),
        _ptr(new_len), _ptr(kl), B, h_kv, T_max, T_out, budget, int(sink), int(recent), d, dt, _stream()))
    return kept, new_len


def kv_evict_paged(k_pages: torch.Tensor, v_pages: torch.Tensor, block_table, weights: torch.Tensor, budget: int,
                   *, kv_len=None, sink: int = 0, recent: int = 0, block_table_out=None, weights_out=None,
                   kept=None):
    """``kv_evict`` over a paged cache: in place, or with ``block_table_out`` (B, max_pages_out) into other pages
    of the same pools (each column another page, or the sequence's own page of that column)."""
    num_pages, h_kv, page_size, d = _pool_shape(k_pages, v_pages)
    _need_cuda(k_pages, v_pages)
    B = weights.shape[0]
    bt = _block_table(block_table, B, k_pages.device)
    bo = None if block_table_out is None else _block_table(block_table_out, B, k_pages.device)
    max_out = bt.shape[1] if bo is None else bo.shape[1]
    dt, budget, weights_out, kept, new_len, kl = _evict_args(k_pages, v_pages, weights, B, h_kv, bt.shape[1] * page_size,
                                                             max_out * page_size, budget, kv_len, weights_out, kept)
    _check("kv_evict_paged", _lib.kv_evict_paged(
        _ptr(k_pages), _ptr(v_pages), _ptr(bt), _ptr(bo), _ptr(weights), _ptr(weights_out), _ptr(kept), _ptr(new_len),
        _ptr(kl), B, h_kv, num_pages, page_size, bt.shape[1], max_out, budget, int(sink), int(recent), d, dt,
        _stream()))
    return kept, new_len
