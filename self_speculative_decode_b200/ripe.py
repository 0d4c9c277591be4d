"""Python binding of libripe.so: same names as the C ABI in include/ripe.h.

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity and passed as raw device pointers; every step of the work runs in the
library's CUDA kernels.  There is no fallback: if the shared library is missing
or no CUDA device is present, calls raise.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# the library to load: libripe.so, or another build of the same sources (e.g. the debug build
# lib/libripe_debug.so) named by the environment variable RIPE_LIBRARY
LIB_PATH = os.environ.get("RIPE_LIBRARY") or os.path.join(PKG, "lib", "libripe.so")

RIPE_OK, RIPE_EINVAL, RIPE_ENOMEM, RIPE_ECAPACITY, RIPE_ESTATE, RIPE_ECUDA = 0, -1, -2, -3, -4, -5
RIPE_WINDOW_QUERY_RELATIVE, RIPE_WINDOW_CACHE_RELATIVE = 0, 1
RIPE_DEVERR_WAIT_TIMEOUT, RIPE_DEVERR_CAPACITY, RIPE_DEVERR_ACCEPT, RIPE_DEVERR_BOUNDS = 1, 2, 4, 8
RIPE_BUILD_DEBUG = 1
RIPE_CONSUMER_DEFAULT, RIPE_CONSUMER_MMA, RIPE_CONSUMER_TC = 0, 1, 2

# exported entry points (kept in step with include/ripe.h; a CPU test checks both)
EXPORTS = (
    "ripe_cache_alloc", "ripe_cache_free", "ripe_load_prefix", "ripe_append_block",
    "ripe_verify_attn", "ripe_commit", "ripe_commit_device", "ripe_sync_lengths",
    "ripe_cache_stats", "ripe_cache_export", "ripe_get_device_error", "ripe_launch_count",
    "ripe_strerror", "ripe_verify_attn_static", "ripe_verify_attn_wave", "ripe_append_verify",
    "ripe_draft_attn", "ripe_draft_attn_window", "ripe_build_info", "ripe_set_verify_consumer",
    "ripe_get_verify_consumer", "ripe_cache_alloc_q8", "ripe_cache_kv_bits", "ripe_cache_export_q8",
    "ripe_set_scores", "ripe_append_block_rope", "ripe_rotate_block", "ripe_append_rope_static",
)
RIPE_ESCRATCH = -6
RIPE_STATIC_SCRATCH_BYTES = 4 << 20


class RipeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} ({status})")


class _Stats(ctypes.Structure):
    _fields_ = [("stored_position_planes", ctypes.c_int64), ("full_position_planes", ctypes.c_int64),
                ("kv_bytes", ctypes.c_int64), ("scratch_bytes", ctypes.c_int64),
                ("deep_rows", ctypes.c_int32), ("ring_slots", ctypes.c_int32),
                ("block_len", ctypes.c_int32), ("lengths_synced", ctypes.c_int32)]


class CacheView(ctypes.Structure):
    """ripe_cache_view: caller-owned cache buffers for ripe_verify_attn_static."""
    _fields_ = [(name, ctypes.c_int32) for name in
                ("batch", "layers", "q_heads", "kv_heads", "head_dim", "loops", "window", "max_T",
                 "max_B", "window_mode", "block_len")] + \
               [(name, ctypes.c_void_p) for name in ("k_deep", "v_deep", "k_ring", "v_ring", "lengths")]


class Rope(ctypes.Structure):
    """ripe_rope: cos and sin tables of the position rotation (RotaryTable holds the tensors)."""
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p)] + \
               [(name, ctypes.c_int32) for name in ("positions", "rotary_dim", "interleaved")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libripe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m self_speculative_decode_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        i32p = ctypes.POINTER(ctypes.c_int32)
        sig = {
            "ripe_cache_alloc": ([i] * 10 + [ctypes.POINTER(vp)], i),
            "ripe_cache_free": ([vp], i),
            "ripe_load_prefix": ([vp, i, i, i32p, vp, vp, i64, vp], i),
            "ripe_append_block": ([vp, i, i, i, vp, vp, vp], i),
            "ripe_verify_attn": ([vp, i, i, vp, vp, vp, ctypes.c_float, vp], i),
            "ripe_commit": ([vp, i32p, vp], i),
            "ripe_commit_device": ([vp, vp, vp], i),
            "ripe_sync_lengths": ([vp, i32p, vp], i),
            "ripe_cache_stats": ([vp, ctypes.POINTER(_Stats)], i),
            "ripe_cache_export": ([vp, i, i, vp, vp, vp, vp], i),
            "ripe_get_device_error": ([vp, ctypes.POINTER(ctypes.c_uint32), vp], i),
            "ripe_launch_count": ([vp], i64),
            "ripe_build_info": ([], i),
            "ripe_set_verify_consumer": ([i], i),
            "ripe_get_verify_consumer": ([], i),
            "ripe_strerror": ([i], ctypes.c_char_p),
            "ripe_verify_attn_static": ([ctypes.POINTER(CacheView), i, i, vp, vp, vp, ctypes.c_float, vp, vp], i),
            "ripe_verify_attn_wave": ([vp, i, i32p, vp, vp, vp, ctypes.c_float, vp], i),
            "ripe_append_verify": ([vp, i, i, i, vp, vp, vp, vp, vp, ctypes.c_float, vp], i),
            "ripe_draft_attn": ([vp, i, i, i, vp, vp, vp, vp, vp, ctypes.c_float, vp], i),
            "ripe_draft_attn_window": ([vp, i, i, i, i, i, vp, vp, vp, vp, vp, ctypes.c_float, vp], i),
            "ripe_cache_alloc_q8": ([i] * 10 + [ctypes.POINTER(vp)], i),
            "ripe_cache_kv_bits": ([vp], i),
            "ripe_cache_export_q8": ([vp, i, i, vp, vp, vp, vp, vp], i),
            "ripe_set_scores": ([vp, ctypes.c_float, ctypes.POINTER(ctypes.c_float), vp], i),
            "ripe_append_block_rope": ([vp, i, i, i, vp, vp, i64, vp, i64, vp, ctypes.POINTER(Rope), vp], i),
            "ripe_rotate_block": ([vp, i, i, vp, i64, vp, vp, i64, vp, ctypes.POINTER(Rope), vp], i),
            "ripe_append_rope_static": ([ctypes.POINTER(CacheView), i, i, vp, vp, i64, vp, i64, vp,
                                         ctypes.POINTER(Rope), vp, vp], i),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().ripe_strerror(status).decode()


def _check(status: int, where: str):
    if status != RIPE_OK:
        raise RipeError(status, where)


_torch = None


def _load_torch():
    """torch, imported at the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _stream(stream):
    """The raw handle of a stream: the current one, a torch stream or an int."""
    if stream is None:
        torch = _torch or _load_torch()
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _made(make, stream, device):
    """make() with the call's stream current: a tensor belongs to the stream that is current when it is allocated, and
    memory that another one still uses, or clears, is no place for this call's results."""
    if stream is None:
        return make()
    torch = _torch or _load_torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return make()


def _dev(t, dtype, shape, name, device=None):
    """Address of a contiguous CUDA tensor of this dtype and (unless None) shape, on the device with this number."""
    torch = _torch or _load_torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the cache on cuda:{device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, dtype, shape, name):
    """Address and token stride (elements) of a [N][B][heads][d] tensor whose heads are packed and whose tokens
    lie at one stride, as a part of a projection's output does."""
    torch = _torch or _load_torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    N, B, H, d = shape
    if t.is_contiguous():
        return t.data_ptr(), H * d
    s = t.stride()
    # the stride of a dimension of one element says nothing
    ld = s[1] if B > 1 else s[0] if N > 1 else H * d
    if s[3] != 1 or (H > 1 and s[2] != d) or (N > 1 and B > 1 and s[0] != B * ld):
        raise ValueError(f"{name} must have packed heads and evenly spaced tokens, got strides {tuple(s)}")
    return t.data_ptr(), ld


def _ints(values, n):
    arr = (ctypes.c_int32 * n)(*[int(x) for x in values])
    if len(values) != n:
        raise ValueError(f"expected {n} values")
    return arr


# ------------------------------------------------------------------ C-ABI mirrors
def ripe_cache_alloc(batch, layers, q_heads, kv_heads, head_dim, loops, window, max_T, max_B,
                     window_mode=RIPE_WINDOW_QUERY_RELATIVE):
    h = ctypes.c_void_p()
    _check(lib().ripe_cache_alloc(batch, layers, q_heads, kv_heads, head_dim, loops, window, max_T,
                                  max_B, window_mode, ctypes.byref(h)), "ripe_cache_alloc")
    return h


def ripe_cache_free(h):
    _check(lib().ripe_cache_free(h), "ripe_cache_free")


def ripe_load_prefix(h, layer, plane, T, k, v, ld_t, stream=None):
    n = len(T)
    _check(lib().ripe_load_prefix(h, layer, plane, _ints(T, n), k, v,
                                  ld_t, _stream(stream)), "ripe_load_prefix")


def ripe_append_block(h, layer, r, B, k, v, stream=None):
    _check(lib().ripe_append_block(h, layer, r, B, k, v, _stream(stream)),
           "ripe_append_block")


def ripe_verify_attn(h, layer, r, q, out, lse=None, scale=1.0, stream=None):
    _check(lib().ripe_verify_attn(h, layer, r, q, out,
                                  lse or None, float(scale), _stream(stream)),
           "ripe_verify_attn")


def ripe_append_verify(h, layer, r, B, k, v, q, out, lse=None, scale=1.0, stream=None):
    _check(lib().ripe_append_verify(h, layer, r, B, k, v, q,
                                    out, lse or None, float(scale),
                                    _stream(stream)), "ripe_append_verify")


def ripe_draft_attn(h, layer, r, j, k, v, q, out, lse=None, scale=1.0, stream=None):
    _check(lib().ripe_draft_attn(h, layer, r, j, k, v, q,
                                 out, lse or None, float(scale),
                                 _stream(stream)), "ripe_draft_attn")


def ripe_draft_attn_window(h, layer, r, j, sink, window, k, v, q, out, lse=None, scale=1.0, stream=None):
    _check(lib().ripe_draft_attn_window(h, layer, r, j, int(sink), int(window), k, v,
                                        q, out, lse or None,
                                        float(scale), _stream(stream)), "ripe_draft_attn_window")


def ripe_verify_attn_wave(h, layer, loop_of_position, q, out, lse=None, scale=1.0, stream=None):
    _check(lib().ripe_verify_attn_wave(h, layer, _ints(loop_of_position, len(loop_of_position)),
                                       q, out, lse or None,
                                       float(scale), _stream(stream)), "ripe_verify_attn_wave")


def ripe_commit(h, accepted_len, stream=None):
    _check(lib().ripe_commit(h, _ints(accepted_len, len(accepted_len)), _stream(stream)), "ripe_commit")


def ripe_commit_device(h, accepted_ptr, stream=None):
    _check(lib().ripe_commit_device(h, accepted_ptr, _stream(stream)), "ripe_commit_device")


def ripe_sync_lengths(h, n, stream=None):
    out = (ctypes.c_int32 * n)()
    _check(lib().ripe_sync_lengths(h, out, _stream(stream)), "ripe_sync_lengths")
    return list(out)


def ripe_cache_stats(h):
    st = _Stats()
    _check(lib().ripe_cache_stats(h, ctypes.byref(st)), "ripe_cache_stats")
    return {name: getattr(st, name) for name, _ in _Stats._fields_}


def ripe_cache_export(h, n, layer, k_out, v_out, present, stream=None):
    _check(lib().ripe_cache_export(h, n, layer, k_out, v_out,
                                   present, _stream(stream)), "ripe_cache_export")


def ripe_get_device_error(h, stream=None):
    e = ctypes.c_uint32()
    _check(lib().ripe_get_device_error(h, ctypes.byref(e), _stream(stream)), "ripe_get_device_error")
    return e.value


def ripe_verify_attn_static(view, layer, r, q, out, lse=None, scale=1.0, device_error=None, stream=None):
    """Allocation-free verify over caller-owned buffers (see include/ripe.h); pointers are ints."""
    _check(lib().ripe_verify_attn_static(ctypes.byref(view), layer, r, q, out,
                                         lse or None, float(scale),
                                         device_error or None, _stream(stream)),
           "ripe_verify_attn_static")


def ripe_cache_alloc_q8(batch, layers, q_heads, kv_heads, head_dim, loops, window, max_T, max_B,
                        window_mode=RIPE_WINDOW_QUERY_RELATIVE):
    h = ctypes.c_void_p()
    _check(lib().ripe_cache_alloc_q8(batch, layers, q_heads, kv_heads, head_dim, loops, window, max_T,
                                     max_B, window_mode, ctypes.byref(h)), "ripe_cache_alloc_q8")
    return h


def ripe_cache_kv_bits(h):
    bits = lib().ripe_cache_kv_bits(h)
    _check(bits if bits < 0 else RIPE_OK, "ripe_cache_kv_bits")
    return bits


def ripe_cache_export_q8(h, n, layer, k_out, v_out, k_scale, v_scale, stream=None):
    _check(lib().ripe_cache_export_q8(h, n, layer, k_out, v_out,
                                      k_scale, v_scale, _stream(stream)),
           "ripe_cache_export_q8")


def ripe_set_scores(h, softcap=0.0, slopes=None, stream=None):
    """slopes: a sequence of q_heads floats (the caller checks the length), or None."""
    arr = None if slopes is None else (ctypes.c_float * len(slopes))(*[float(x) for x in slopes])
    _check(lib().ripe_set_scores(h, float(softcap), arr, _stream(stream)), "ripe_set_scores")


def ripe_append_block_rope(h, layer, r, B, k, v, ld_kv, q, ld_q, q_out, rope, stream=None):
    _check(lib().ripe_append_block_rope(h, layer, r, B, k, v, ld_kv,
                                        q or None, ld_q, q_out or None,
                                        ctypes.byref(rope), _stream(stream)), "ripe_append_block_rope")


def ripe_rotate_block(h, j, B, k, ld_k, k_out, q, ld_q, q_out, rope, stream=None):
    _check(lib().ripe_rotate_block(h, j, B, k or None, ld_k, k_out or None,
                                   q or None, ld_q, q_out or None, ctypes.byref(rope),
                                   _stream(stream)), "ripe_rotate_block")


def ripe_append_rope_static(view, layer, r, k, v, ld_kv, q, ld_q, q_out, rope, device_error, stream=None):
    """Append over caller-owned buffers (see include/ripe.h); pointers are ints, rope a Rope or None."""
    _check(lib().ripe_append_rope_static(ctypes.byref(view), layer, r, k, v, ld_kv,
                                         q or None, ld_q, q_out or None,
                                         None if rope is None else ctypes.byref(rope),
                                         device_error, _stream(stream)), "ripe_append_rope_static")


def ripe_launch_count(h):
    return lib().ripe_launch_count(h)


def ripe_build_info():
    return lib().ripe_build_info()


def ripe_set_verify_consumer(consumer):
    """Select the consumer of verification launches with 9..64 query rows per kv head (process-wide);
    returns the previous choice."""
    prev = lib().ripe_set_verify_consumer(int(consumer))
    _check(prev if prev < 0 else RIPE_OK, "ripe_set_verify_consumer")
    return prev


def ripe_get_verify_consumer():
    return lib().ripe_get_verify_consumer()


# ------------------------------------------------------------------ tensor-level wrapper
class RotaryTable:
    """cos and sin of the position rotation: fp32 [positions][rotary_dim / 2], contiguous, on the cache's device.

    ``interleaved``: a pair is elements 2 i and 2 i + 1 of a head; else i and rotary_dim / 2 + i."""

    def __init__(self, cos, sin, interleaved=False):
        torch = _torch or _load_torch()
        if cos.dim() != 2:
            raise ValueError("cos must be [positions][rotary_dim / 2]")
        self.cos, self.sin = cos, sin  # the struct below points into them
        self.rope = Rope(cos=_dev(cos, torch.float32, None, "cos"),
                         sin=_dev(sin, torch.float32, cos.shape, "sin"), positions=cos.shape[0],
                         rotary_dim=2 * cos.shape[1], interleaved=1 if interleaved else 0)


def append_rope_static(view, layer, r, k, v, q=None, table=None, q_out=None, device_error=None, stream=None):
    """ripe_append_rope_static with tensors: k, v [N][B][kvH][d] and q [N][B][Hq][d] (tokens may be strided) into the
    ring of ``view`` (a CacheView) and into ``q_out``, which is returned.  ``table``: a RotaryTable, or None to copy
    without rotating.  ``device_error``: an int32 tensor of one element that collects RIPE_DEVERR_* bits."""
    torch = _torch or _load_torch()
    N, B = view.batch, view.block_len
    kp, ld_kv = _rows(k, torch.bfloat16, (N, B, view.kv_heads, view.head_dim), "k")
    vp, ld_v = _rows(v, torch.bfloat16, (N, B, view.kv_heads, view.head_dim), "v")
    if ld_v != ld_kv:
        raise ValueError("k and v must have the same token stride")
    if device_error is None:
        raise ValueError("device_error must be given")
    here = torch.cuda.current_device()
    for t in (k, v, q, q_out, device_error, table and table.cos, table and table.sin):
        if t is not None and t.get_device() != here:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{here}")
    qp, ld_q, qo = None, 0, None
    if q is not None:
        shape = (N, B, view.q_heads, view.head_dim)
        qp, ld_q = _rows(q, torch.bfloat16, shape, "q")
        if q_out is None:
            q_out = _made(lambda: torch.empty(shape, dtype=torch.bfloat16, device=q.device), stream, here)
        qo = _dev(q_out, torch.bfloat16, shape, "q_out")
    ripe_append_rope_static(view, layer, r, kp, vp, ld_kv, qp, ld_q, qo, None if table is None else table.rope,
                            _dev(device_error, torch.int32, (1,), "device_error"), stream)
    return q_out


class RipeCache:
    """A RIPE cache on the current CUDA device, driven with torch tensors.

    A call runs on ``stream`` (a torch stream, or its handle as an int), or on the current stream of the cache's device;
    what it allocates for its results belongs to that stream.

    ``kv_bits``: 16, or 8 to hold the deepest-plane region in 8 bits with a scale for each 64 positions.

    Shapes (bf16, contiguous, on the cache's device):
      prefix plane  k, v [N][kvH][ld_t][d]
      block plane   k, v [N][B][kvH][d]
      queries       q, out [N][B][Hq][d]; lse fp32 [N][B][Hq]
    """

    def __init__(self, batch, layers, q_heads, kv_heads, head_dim, loops, window, max_T, max_B,
                 window_mode=RIPE_WINDOW_QUERY_RELATIVE, kv_bits=16):
        torch = _load_torch()
        if kv_bits not in (8, 16):
            raise ValueError("kv_bits must be 8 or 16")
        if not torch.cuda.is_available():
            raise RuntimeError("RipeCache needs a CUDA device")
        self.N, self.L, self.Hq, self.kvH, self.d = batch, layers, q_heads, kv_heads, head_dim
        self.R, self.W, self.max_T, self.max_B, self.mode = loops, window, max_T, max_B, window_mode
        self.kv_bits, self.device = kv_bits, torch.cuda.current_device()
        self.handle = (ripe_cache_alloc if kv_bits == 16 else ripe_cache_alloc_q8)(
            batch, layers, q_heads, kv_heads, head_dim, loops, window, max_T, max_B, window_mode)

    def _on(self, stream):
        """The stream of a call: the one given, or the current one of the cache's device."""
        return _torch._C._cuda_getCurrentRawStream(self.device) if stream is None else stream

    def _here(self, *tensors):
        for t in tensors:
            if t is not None and t.get_device() != self.device:
                raise ValueError(f"a tensor is on {t.device}, the cache on cuda:{self.device}")

    def close(self):
        if self.handle is not None and self.handle.value:
            ripe_cache_free(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load_prefix(self, layer, plane, T, k, v, stream=None):
        torch = _torch or _load_torch()
        ld_t = k.shape[2]
        shape = (self.N, self.kvH, ld_t, self.d)
        ripe_load_prefix(self.handle, layer, plane, list(T), _dev(k, torch.bfloat16, shape, "k", self.device),
                         _dev(v, torch.bfloat16, shape, "v", self.device), ld_t, self._on(stream))

    def append_block(self, layer, r, k, v, stream=None):
        torch = _torch or _load_torch()
        B = k.shape[1]
        shape = (self.N, B, self.kvH, self.d)
        ripe_append_block(self.handle, layer, r, B, _dev(k, torch.bfloat16, shape, "k", self.device),
                          _dev(v, torch.bfloat16, shape, "v", self.device), self._on(stream))

    def set_scores(self, softcap=0.0, slopes=None, stream=None):
        """Capped scores (softcap > 0) and a bias -slopes[h] * distance (Hq floats) in every later attention call."""
        if slopes is not None:
            slopes = slopes.tolist() if hasattr(slopes, "tolist") else list(slopes)
            if len(slopes) != self.Hq:
                raise ValueError(f"expected {self.Hq} slopes")
        ripe_set_scores(self.handle, softcap, slopes, self._on(stream))

    def append_block_rope(self, layer, r, k, v, table, q=None, q_out=None, stream=None):
        """append_block with k, and q if given, rotated by their positions; k, v and q may be parts of one projection's
        output (tokens strided).  Returns q_out."""
        torch = _torch or _load_torch()
        B = k.shape[1]
        kp, ld_kv = _rows(k, torch.bfloat16, (self.N, B, self.kvH, self.d), "k")
        vp, ld_v = _rows(v, torch.bfloat16, (self.N, B, self.kvH, self.d), "v")
        if ld_v != ld_kv:
            raise ValueError("k and v must have the same token stride")
        qp, ld_q, q_out, qo = self._rotated(q, q_out, B, self.Hq, "q", stream)
        self._here(k, v, q, q_out, table.cos, table.sin)
        ripe_append_block_rope(self.handle, layer, r, B, kp, vp, ld_kv, qp, ld_q, qo, table.rope, self._on(stream))
        return q_out

    def rotate_block(self, j, table, k=None, q=None, k_out=None, q_out=None, stream=None):
        """k [N][B][kvH][d] and q [N][B][Hq][d] of block positions j .. j + B - 1 rotated, for the draft calls and
        append_verify; returns (k_out, q_out)."""
        B = (k if k is not None else q).shape[1]
        kp, ld_k, k_out, ko = self._rotated(k, k_out, B, self.kvH, "k", stream)
        qp, ld_q, q_out, qo = self._rotated(q, q_out, B, self.Hq, "q", stream)
        self._here(k, q, k_out, q_out, table.cos, table.sin)
        ripe_rotate_block(self.handle, j, B, kp, ld_k, ko, qp, ld_q, qo, table.rope, self._on(stream))
        return k_out, q_out

    def _rotated(self, x, x_out, B, heads, name, stream):
        torch = _torch or _load_torch()
        if x is None:
            return None, 0, None, None
        shape = (self.N, B, heads, self.d)
        p, ld = _rows(x, torch.bfloat16, shape, name)
        if x_out is None:
            x_out = _made(lambda: torch.empty(shape, dtype=torch.bfloat16, device=x.device), stream, self.device)
        return p, ld, x_out, _dev(x_out, torch.bfloat16, shape, name + "_out")

    def verify_attn(self, layer, r, q, out=None, lse=None, scale=1.0, stream=None):
        torch = _torch or _load_torch()
        B = q.shape[1]
        shape = (self.N, B, self.Hq, self.d)
        qp = _dev(q, torch.bfloat16, shape, "q", self.device)
        if out is None:
            out = _made(lambda: torch.empty_like(q), stream, self.device)  # contiguous, as q
        op = _dev(out, torch.bfloat16, shape, "out", self.device)
        lp = _dev(lse, torch.float32, shape[:3], "lse", self.device) if lse is not None else None
        ripe_verify_attn(self.handle, layer, r, qp, op, lp, scale, self._on(stream))
        return out

    def append_verify(self, layer, r, k, v, q, out=None, lse=None, scale=1.0, stream=None):
        """append_block(layer, r, k, v) + verify_attn(layer, r, q) in one launch."""
        torch = _torch or _load_torch()
        B = q.shape[1]
        kshape = (self.N, B, self.kvH, self.d)
        shape = (self.N, B, self.Hq, self.d)
        kp = _dev(k, torch.bfloat16, kshape, "k", self.device)
        vp = _dev(v, torch.bfloat16, kshape, "v", self.device)
        qp = _dev(q, torch.bfloat16, shape, "q", self.device)
        if out is None:
            out = _made(lambda: torch.empty_like(q), stream, self.device)  # contiguous, as q
        op = _dev(out, torch.bfloat16, shape, "out", self.device)
        lp = _dev(lse, torch.float32, shape[:3], "lse", self.device) if lse is not None else None
        ripe_append_verify(self.handle, layer, r, B, kp, vp, qp, op, lp, scale, self._on(stream))
        return out

    def draft_attn(self, layer, r, j, k, v, q, out=None, lse=None, scale=1.0, stream=None, sink=None,
                   window=None):
        """Draft step: write plane r of block position j (k, v [N][1][kvH][d]) and attend its
        query q [N][1][Hq][d] over keys up to that position; with ``sink`` / ``window`` only
        over the first ``sink`` keys and the last ``window`` + 1 (windowed draft attention)."""
        torch = _torch or _load_torch()
        kshape = (self.N, 1, self.kvH, self.d)
        shape = (self.N, 1, self.Hq, self.d)
        kp = _dev(k, torch.bfloat16, kshape, "k", self.device)
        vp = _dev(v, torch.bfloat16, kshape, "v", self.device)
        qp = _dev(q, torch.bfloat16, shape, "q", self.device)
        if out is None:
            out = _made(lambda: torch.empty_like(q), stream, self.device)  # contiguous, as q
        op = _dev(out, torch.bfloat16, shape, "out", self.device)
        lp = _dev(lse, torch.float32, shape[:3], "lse", self.device) if lse is not None else None
        if sink is None and window is None:
            ripe_draft_attn(self.handle, layer, r, j, kp, vp, qp, op, lp, scale, self._on(stream))
        else:
            ripe_draft_attn_window(self.handle, layer, r, j, 0 if sink is None else sink,
                                   (1 << 30) if window is None else window, kp, vp, qp, op, lp, scale, self._on(stream))
        return out

    def verify_attn_wave(self, layer, loop_of_position, q, out=None, lse=None, scale=1.0, stream=None):
        """Block position j verified at loop loop_of_position[j] (one pass over the deepest plane)."""
        torch = _torch or _load_torch()
        B = q.shape[1]
        shape = (self.N, B, self.Hq, self.d)
        qp = _dev(q, torch.bfloat16, shape, "q", self.device)
        if out is None:
            out = _made(lambda: torch.empty_like(q), stream, self.device)  # contiguous, as q
        op = _dev(out, torch.bfloat16, shape, "out", self.device)
        lp = _dev(lse, torch.float32, shape[:3], "lse", self.device) if lse is not None else None
        ripe_verify_attn_wave(self.handle, layer, list(loop_of_position), qp, op, lp, scale, self._on(stream))
        return out

    def commit(self, accepted_len, stream=None):
        ripe_commit(self.handle, list(accepted_len), self._on(stream))

    def commit_device(self, accepted, stream=None):
        torch = _torch or _load_torch()
        ripe_commit_device(self.handle, _dev(accepted, torch.int32, (self.N,), "accepted", self.device), self._on(stream))

    def sync_lengths(self, stream=None):
        return ripe_sync_lengths(self.handle, self.N, self._on(stream))

    def stats(self):
        return ripe_cache_stats(self.handle)

    def export(self, n, layer, stream=None):
        """Logical view of sequence n, layer: (k, v [R][kvH][Tv][d] bf16, present [R][Tv] uint8)."""
        torch = _torch or _load_torch()
        st = self.stats()
        if not st["lengths_synced"]:
            raise RipeError(RIPE_ESTATE, "export")
        Tv = self.sync_lengths(stream)[n] + st["block_len"]
        dev = torch.device("cuda", self.device)
        k, v, present = _made(lambda: (*(torch.zeros((self.R, self.kvH, Tv, self.d), dtype=torch.bfloat16, device=dev)
                                         for _ in range(2)),
                                       torch.zeros((self.R, Tv), dtype=torch.uint8, device=dev)), stream, self.device)
        if Tv:
            ripe_cache_export(self.handle, n, layer, k.data_ptr(), v.data_ptr(), present.data_ptr(), self._on(stream))
        return k, v, present

    def export_q8(self, n, layer, stream=None):
        """8-bit blocks of sequence n, layer: k, v int8 [kvH][D][d] and their scales fp32 [kvH][D / 64]."""
        torch = _torch or _load_torch()
        if not self.stats()["lengths_synced"]:
            raise RipeError(RIPE_ESTATE, "export_q8")
        blocks = max(0, self.sync_lengths(stream)[n] - self.W) // 64
        dev = torch.device("cuda", self.device)
        k, v, ks, vs = _made(lambda: [torch.empty((self.kvH, 64 * blocks, self.d), dtype=torch.int8, device=dev)
                                      for _ in range(2)] +
                                     [torch.empty((self.kvH, blocks), dtype=torch.float32, device=dev) for _ in range(2)],
                             stream, self.device)
        if blocks or self.kv_bits != 8:
            ripe_cache_export_q8(self.handle, n, layer, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), self._on(stream))
        return k, v, ks, vs

    def device_error(self, stream=None):
        return ripe_get_device_error(self.handle, self._on(stream))

    def launch_count(self):
        return ripe_launch_count(self.handle)
