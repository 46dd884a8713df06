"""Thin ctypes binding of the C ABI in include/oscar.h (argument marshalling only).

Every computation runs in the CUDA library; this module only converts Python
objects (torch tensors, numpy arrays, ints) into the pointers and sizes the C
functions take, and raises ``OscarError`` on a non-OK status.  Importing it
loads the library and fails loudly if it has not been built.
"""
from __future__ import annotations

import ctypes
import operator
import os
import warnings
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_uint64, c_void_p

import numpy as np

from .build import LIB, calls_path

OSCAR_OK = 0
OSCAR_ERR_INVALID_ARG = 1
OSCAR_ERR_OUT_OF_PAGES = 2
OSCAR_ERR_STATE = 3
OSCAR_ERR_CUDA = 4
OSCAR_ERR_TIMEOUT = 5
OSCAR_ERR_DEVICE_CHECK = 6
OSCAR_ERR_DRY_RUN = 7
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "OUT_OF_PAGES", 3: "STATE", 4: "CUDA", 5: "TIMEOUT",
                6: "DEVICE_CHECK", 7: "DRY_RUN"}

HEAD_DIM = 128
RECORD_BYTES = 4608
BF16_PAGES_PER_REQUEST = 5


class oscar_cache_config(ctypes.Structure):
    _fields_ = [("num_layers", c_int32), ("num_q_heads", c_int32), ("num_kv_heads", c_int32),
                ("head_dim", c_int32), ("sink_tokens", c_int32), ("recent_tokens", c_int32),
                ("page_tokens", c_int32), ("group_size", c_int32), ("max_requests", c_int32),
                ("max_pages_per_request", c_int32), ("num_int2_pages", c_int64), ("num_bf16_pages", c_int64),
                ("softmax_scale", c_float), ("page_perm_seed", c_uint64)]


class oscar_cache_layout(ctypes.Structure):
    _fields_ = [(name, c_size_t) for name in (
        "total_bytes", "int2_pool_offset", "int2_layer_stride", "int2_page_stride", "int2_record_bytes",
        "bf16_pool_offset", "bf16_layer_stride", "bf16_page_stride", "bf16_record_bytes",
        "rot_k_offset", "rot_v_offset", "rot_kt_offset", "rot_vt_offset", "rot_colnorm_offset",
        "tau_k_offset", "tau_v_offset",
        "hist_pt_offset", "bf16_pt_offset", "error_word_offset", "decode_count_offset", "decode_flag_offset")]


class oscar_rope(ctypes.Structure):
    _fields_ = [("table", c_void_p), ("length", c_int32), ("dim", c_int32), ("interleaved", c_int32)]


OSCAR_F32, OSCAR_BF16 = 0, 1


class OscarError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_P = c_void_p
_SIGNATURES = {
    "oscar_version": (c_char_p, []),
    "oscar_cache_device_bytes": (c_size_t, [POINTER(oscar_cache_config)]),
    "oscar_cache_create": (c_int32, [POINTER(oscar_cache_config), _P, c_size_t, _P, _P, POINTER(c_float),
                                     POINTER(c_float), _P, POINTER(_P)]),
    "oscar_cache_destroy": (c_int32, [_P]),
    "oscar_cache_get_layout": (c_int32, [_P, POINTER(oscar_cache_layout)]),
    "oscar_request_open": (c_int32, [_P, _P, POINTER(c_int32)]),
    "oscar_request_fork": (c_int32, [_P, c_int32, c_int64, _P, POINTER(c_int32)]),
    "oscar_request_close": (c_int32, [_P, c_int32]),
    "oscar_request_length": (c_int32, [_P, c_int32, c_int32, POINTER(c_int64), POINTER(c_int64)]),
    "oscar_request_pages": (c_int32, [_P, c_int32, POINTER(c_int32), c_int32, POINTER(c_int32), POINTER(c_int32)]),
    "oscar_cache_free_pages": (c_int32, [_P, POINTER(c_int64), POINTER(c_int64)]),
    "oscar_prefill_quantize": (c_int32, [_P, c_int32, c_int32, _P, _P, c_int64, _P]),
    "oscar_append": (c_int32, [_P, c_int32, c_int32, POINTER(c_int32), _P, _P, _P]),
    "oscar_demote": (c_int32, [_P, c_int32, c_int32, POINTER(c_int32), _P]),
    "oscar_demote_layers": (c_int32, [_P, c_int32, c_int32, c_int32, POINTER(c_int32), _P]),
    "oscar_decode_workspace_bytes": (c_int32, [_P, c_int32, POINTER(c_int32), POINTER(c_size_t)]),
    "oscar_decode_attention": (c_int32, [_P, c_int32, c_int32, POINTER(c_int32), _P, _P, _P, c_size_t, _P]),
    "oscar_decode_attention_noalloc": (c_int32, [_P, c_int32, c_int32, POINTER(c_int32), _P, _P, _P]),
    "oscar_decode_step": (c_int32, [_P, c_int32, c_int32, POINTER(c_int32), _P, _P, _P, _P, _P, c_size_t, _P]),
    "oscar_cache_check": (c_int32, [_P, _P]),
    "oscar_debug_decode_hooks": (c_int32, [_P, ctypes.c_uint32, c_int32]),
    "oscar_last_error": (c_char_p, [_P]),
    "oscar_bf16_decode_workspace_bytes": (c_size_t, [c_int32, POINTER(c_int32), c_int32, c_int32]),
    "oscar_bf16_decode": (c_int32, [_P, c_int64, _P, c_int32, POINTER(c_int32), c_int32, c_int32, c_int32, c_float,
                                    _P, _P, _P, c_size_t, _P]),
    "oscar_bf16_append": (c_int32, [_P, c_int64, _P, c_int32, POINTER(c_int32), POINTER(c_int32), c_int32, c_int32,
                                    c_int32, POINTER(oscar_rope), _P, c_int64, _P, c_int64, _P, c_int64, _P, _P, _P]),
    "oscar_int4_append": (c_int32, [_P, c_int64, _P, c_int32, POINTER(c_int32), POINTER(c_int32), c_int32, c_int32,
                                    c_int32, c_int32, POINTER(oscar_rope), _P, c_int64, _P, c_int64, _P, c_int64, _P,
                                    _P, _P]),
    "oscar_int4_read": (c_int32, [_P, c_int64, _P, c_int32, POINTER(c_int32), POINTER(c_int32), c_int32, c_int32,
                                  c_int32, _P, _P, c_int32, _P, _P]),
    "oscar_attention_workspace_bytes": (c_size_t, [c_int32, POINTER(c_int32), c_int32, c_int32]),
    "oscar_window_attention": (c_int32, [_P, c_int64, _P, c_int32, POINTER(c_int32), POINTER(c_int32), c_int32, c_int32,
                                         c_int32, c_int32, c_int32, c_float, _P, c_int64, _P, c_int32, _P, _P, _P,
                                         c_size_t, _P]),
    "oscar_int4_attention": (c_int32, [_P, c_int64, _P, c_int32, POINTER(c_int32), POINTER(c_int32), c_int32, c_int32,
                                       c_int32, c_int32, c_int32, c_int32, c_float, _P, c_int64, _P, c_int32, _P, _P,
                                       _P, c_size_t, _P]),
    "oscar_paged_last_error": (c_char_p, []),
}

_lib = None


def load(path: str = LIB) -> ctypes.CDLL:
    """Load the CUDA library (once); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing: run bit_rotated_kv_decode_gb300.build.build()")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGNATURES)


def make_config(num_layers, num_q_heads, num_kv_heads, max_requests, max_pages_per_request, num_int2_pages,
                num_bf16_pages=0, softmax_scale=0.0, page_perm_seed=0, group_size=128) -> oscar_cache_config:
    return oscar_cache_config(num_layers, num_q_heads, num_kv_heads, HEAD_DIM, 64, 256, 64, group_size, max_requests,
                              max_pages_per_request, num_int2_pages, num_bf16_pages, softmax_scale, page_perm_seed)


def _ptr(t) -> int | None:
    """Device address of a dense row-major tensor (the C ABI takes no strides)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise OscarError(OSCAR_ERR_INVALID_ARG, "tensor must be contiguous (dense row-major)")
    return t.data_ptr()


def _stream_ptr(stream) -> int | None:
    if stream is None:
        import torch
        if not torch.cuda.is_available():
            return None
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class OscarCache:
    """Owner of one cache handle and its device buffer (a torch uint8 tensor)."""

    def __init__(self, cfg: oscar_cache_config, rot_k=None, rot_v=None, tau_k=None, tau_v=None,
                 device="cuda", stream=None, dry_run: bool = False):
        import torch
        self.lib = load()
        self.cfg = cfg
        self.dry = dry_run
        self.bytes = self.lib.oscar_cache_device_bytes(ctypes.byref(cfg))
        if self.bytes == 0:
            raise OscarError(OSCAR_ERR_INVALID_ARG, "invalid cache configuration")
        lh = cfg.num_layers * cfg.num_kv_heads
        tk = np.ascontiguousarray(np.asarray(tau_k, dtype=np.float32).reshape(lh))
        tv = np.ascontiguousarray(np.asarray(tau_v, dtype=np.float32).reshape(lh))
        self._tau = (tk, tv)
        self.mem = None
        if not dry_run:
            self.mem = torch.empty(self.bytes + 256, dtype=torch.uint8, device=device)
            off = (-self.mem.data_ptr()) % 256
            self.mem = self.mem[off:off + self.bytes]
            assert rot_k.is_cuda and rot_k.dtype == torch.float32 and rot_k.is_contiguous()
            assert rot_v.is_cuda and rot_v.dtype == torch.float32 and rot_v.is_contiguous()
        handle = c_void_p()
        st = self.lib.oscar_cache_create(ctypes.byref(cfg), _ptr(self.mem), self.bytes, _ptr(rot_k), _ptr(rot_v),
                                         tk.ctypes.data_as(POINTER(c_float)), tv.ctypes.data_as(POINTER(c_float)),
                                         None if dry_run else _stream_ptr(stream), ctypes.byref(handle))
        if st != OSCAR_OK:
            raise OscarError(st, "oscar_cache_create failed")
        self.h = handle

    # -- helpers ----------------------------------------------------------------
    def _check(self, st: int, what: str, allow_dry: bool = False) -> None:
        if st == OSCAR_OK or (allow_dry and st == OSCAR_ERR_DRY_RUN and self.dry):
            return
        raise OscarError(st, f"{what}: {self.lib.oscar_last_error(self.h).decode()}")

    def close_handle(self) -> None:
        if getattr(self, "h", None):
            self.lib.oscar_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close_handle()
        except Exception:
            pass

    def layout(self) -> oscar_cache_layout:
        lay = oscar_cache_layout()
        self._check(self.lib.oscar_cache_get_layout(self.h, ctypes.byref(lay)), "layout")
        return lay

    # -- requests -----------------------------------------------------------------
    def open(self, stream=None) -> int:
        r = c_int32()
        self._check(self.lib.oscar_request_open(self.h, None if self.dry else _stream_ptr(stream), ctypes.byref(r)),
                    "open")
        return r.value

    def fork(self, parent: int, prefix_tokens: int, stream=None) -> int:
        r = c_int32()
        self._check(self.lib.oscar_request_fork(self.h, parent, prefix_tokens,
                                                None if self.dry else _stream_ptr(stream), ctypes.byref(r)), "fork")
        return r.value

    def close(self, req: int) -> None:
        self._check(self.lib.oscar_request_close(self.h, req), "close")

    def length(self, req: int, layer: int):
        t, he = c_int64(), c_int64()
        self._check(self.lib.oscar_request_length(self.h, req, layer, ctypes.byref(t), ctypes.byref(he)), "length")
        return t.value, he.value

    def pages(self, req: int):
        n = c_int32()
        bf = (c_int32 * BF16_PAGES_PER_REQUEST)()
        self._check(self.lib.oscar_request_pages(self.h, req, None, 0, ctypes.byref(n), bf), "pages")
        buf = (c_int32 * max(1, n.value))()
        self._check(self.lib.oscar_request_pages(self.h, req, buf, n.value, ctypes.byref(n), bf), "pages")
        return list(buf)[:n.value], list(bf)

    def free_pages(self):
        a, b = c_int64(), c_int64()
        self._check(self.lib.oscar_cache_free_pages(self.h, ctypes.byref(a), ctypes.byref(b)), "free_pages")
        return a.value, b.value

    # -- write path ---------------------------------------------------------------
    def prefill(self, req: int, layer: int, k, v, n_tokens: int | None = None, stream=None) -> None:
        n = int(k.shape[0]) if n_tokens is None else n_tokens
        self._check(self.lib.oscar_prefill_quantize(self.h, req, layer, _ptr(k), _ptr(v), n,
                                                    None if self.dry else _stream_ptr(stream)), "prefill",
                    allow_dry=True)

    @staticmethod
    def _reqs(reqs):
        arr = (c_int32 * len(reqs))(*[int(r) for r in reqs])
        return arr

    def append(self, layer: int, reqs, k, v, stream=None) -> None:
        arr = self._reqs(reqs)
        self._check(self.lib.oscar_append(self.h, layer, len(reqs), arr, _ptr(k), _ptr(v),
                                          None if self.dry else _stream_ptr(stream)), "append", allow_dry=True)

    def demote(self, layer: int, reqs, stream=None) -> None:
        arr = self._reqs(reqs)
        self._check(self.lib.oscar_demote(self.h, layer, len(reqs), arr, None if self.dry else _stream_ptr(stream)),
                    "demote", allow_dry=True)

    def demote_layers(self, layer_begin: int, layer_end: int, reqs, stream=None) -> None:
        arr = self._reqs(reqs)
        self._check(self.lib.oscar_demote_layers(self.h, layer_begin, layer_end, len(reqs), arr,
                                                 None if self.dry else _stream_ptr(stream)),
                    "demote_layers", allow_dry=True)

    # -- decode -------------------------------------------------------------------
    def workspace_bytes(self, reqs) -> int:
        arr = self._reqs(reqs)
        b = c_size_t()
        self._check(self.lib.oscar_decode_workspace_bytes(self.h, len(reqs), arr, ctypes.byref(b)), "workspace")
        return b.value

    def decode(self, layer: int, reqs, q, out, workspace, stream=None) -> None:
        arr = self._reqs(reqs)
        self._check(self.lib.oscar_decode_attention(self.h, layer, len(reqs), arr, _ptr(q), _ptr(out),
                                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                    _stream_ptr(stream)), "decode")

    def step(self, layer: int, reqs, k, v, q, out, workspace, stream=None) -> None:
        """Append k / v of every request, then decode with q (one fused call)."""
        arr = self._reqs(reqs)
        nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        self._check(self.lib.oscar_decode_step(self.h, layer, len(reqs), arr, _ptr(k), _ptr(v), _ptr(q), _ptr(out),
                                               _ptr(workspace), nbytes, None if self.dry else _stream_ptr(stream)),
                    "decode step", allow_dry=True)

    def decode_noalloc(self, layer: int, reqs, q, out, stream=None) -> None:
        """Decode with the library's fixed static scratch (no workspace argument)."""
        arr = self._reqs(reqs)
        self._check(self.lib.oscar_decode_attention_noalloc(self.h, layer, len(reqs), arr, _ptr(q), _ptr(out),
                                                            None if self.dry else _stream_ptr(stream)),
                    "decode (fixed scratch)", allow_dry=True)

    def check(self, stream=None) -> None:
        self._check(self.lib.oscar_cache_check(self.h, None if self.dry else _stream_ptr(stream)), "device check")

    def debug_decode_hooks(self, wait_limit: int = 100000, hold_copy: int = -1) -> None:
        """Failure-detection hooks of this cache's decode launches (tests only)."""
        self._check(self.lib.oscar_debug_decode_hooks(self.h, wait_limit, hold_copy), "decode hooks")

    # -- views of device memory (for tests and inspection) ------------------------
    def int2_pool(self, layer: int):
        lay = self.layout()
        rec = lay.int2_record_bytes          # 4608 (group 128) or 5120 (group 64)
        n = self.cfg.num_int2_pages * self.cfg.num_kv_heads * rec
        base = lay.int2_pool_offset + layer * lay.int2_layer_stride
        return self.mem[base:base + n].view(self.cfg.num_int2_pages, self.cfg.num_kv_heads, rec)

    def bf16_pool(self, layer: int):
        import torch
        lay = self.layout()
        nb = self.cfg.num_bf16_pages or BF16_PAGES_PER_REQUEST * self.cfg.max_requests
        n = nb * lay.bf16_page_stride
        base = lay.bf16_pool_offset + layer * lay.bf16_layer_stride
        return self.mem[base:base + n].view(torch.int16).view(nb, self.cfg.num_kv_heads, 2, 64, HEAD_DIM)

    def device_page_table(self):
        import torch
        lay = self.layout()
        n = self.cfg.max_requests * self.cfg.max_pages_per_request
        return self.mem[lay.hist_pt_offset:lay.hist_pt_offset + 4 * n].view(torch.int32).view(
            self.cfg.max_requests, self.cfg.max_pages_per_request)


def bf16_decode(kv, page_table, lens, q, out, num_kv_heads: int, scale: float = 0.0, workspace=None, stream=None):
    """Uncompressed BF16 paged decode attention (the baseline): kv bf16
    [pages][Hkv][2][64][128], page_table int32 [n][max_pages] (device), lens host
    ints, q bf16 [n][Hq][128], out fp32 [n][Hq][128].  Returns the workspace."""
    lib = load()
    n, hq = q.shape[0], q.shape[1]
    arr = (c_int32 * n)(*[int(x) for x in lens])
    need = lib.oscar_bf16_decode_workspace_bytes(n, arr, hq, num_kv_heads)
    if need == 0:
        raise OscarError(1, "bf16_decode: arguments outside the supported limits")
    if workspace is None or workspace.numel() < need:
        workspace = new_workspace(need)
    st = lib.oscar_bf16_decode(_ptr(kv), kv.shape[0], _ptr(page_table), page_table.shape[1], arr, n, hq,
                               num_kv_heads, float(scale), _ptr(q), _ptr(out), _ptr(workspace), workspace.numel(),
                               _stream_ptr(stream))
    if st != 0:
        raise OscarError(st, "oscar_bf16_decode failed")
    return workspace


def new_workspace(nbytes: int, device="cuda"):
    """Zeroed, 256-byte aligned device workspace of at least nbytes."""
    import torch
    t = torch.zeros(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-t.data_ptr()) % 256
    return t[off:off + nbytes]


# ---- paged caches: position rotation, windowed attention, 4 bits ----------------
INT4_RECORD_BYTES = {128: 8704, 64: 9216}


def rope_table(length: int, dim: int = HEAD_DIM, theta: float = 10000.0, scale: float = 1.0, device="cuda"):
    """fp32 [length][dim]: cosines, then sines, of position * scale * theta^(-2 i / dim).  The angles are
    taken in float64, so that far positions keep theirs; scale 1 / s stretches the positions by s."""
    import torch
    inv = scale * theta ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64) / dim)
    a = torch.arange(length, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)


def int4_pool(num_pages: int, num_kv_heads: int, group_size: int = 128, device="cuda"):
    """Zeroed 4-bit page pool uint8 [num_pages][num_kv_heads][record]."""
    import torch
    if group_size not in INT4_RECORD_BYTES:
        _refuse("group_size must be 128 or 64")
    return torch.zeros(num_pages, num_kv_heads, INT4_RECORD_BYTES[group_size], dtype=torch.uint8, device=device)


def _refuse(what: str):
    raise OscarError(OSCAR_ERR_INVALID_ARG, what)


def _paged_check(st: int, what: str) -> None:
    if st != OSCAR_OK:
        raise OscarError(st, f"{what}: {load().oscar_paged_last_error().decode()}")


# These calls are made for every layer of a decode step, so they are marshalled in C++
# (csrc/calls.cpp).  What that does not take as it is -- a tensor that fails a check, no
# workspace yet, a stream of its own, lengths that are no list of ints -- goes the same way
# in Python below, which says what is wrong; so does every call where the extension has not
# been built for this torch.
_torch = None
_calls = None


class _NotBuilt:
    """Takes no call, as the extension where it leaves one to Python."""
    append = read = attend = staticmethod(lambda *args: None)


def calls():
    """The extension that marshals the paged calls (loaded once; raises if it has not been built)."""
    global _calls
    if _calls is None or _calls is _NotBuilt:
        import importlib.machinery
        import importlib.util
        path = calls_path()
        if not os.path.exists(path):
            raise RuntimeError(f"extension {path} is missing: run bit_rotated_kv_decode_gb300.build.build()")
        loader = importlib.machinery.ExtensionFileLoader("_oscar_calls", path)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_oscar_calls", loader))
        loader.exec_module(mod)
        lib = load()
        mod.setup(tuple(ctypes.cast(fn, c_void_p).value for fn in (
            lib.oscar_bf16_append, lib.oscar_int4_append, lib.oscar_int4_read, lib.oscar_window_attention,
            lib.oscar_int4_attention)))
        _calls = mod
    return _calls


def _marshal():
    global _calls
    if os.path.exists(calls_path()):
        return calls()
    warnings.warn("the extension that marshals the paged calls is not built for this torch: they are marshalled in "
                  "Python, 9 us a call slower (bit_rotated_kv_decode_gb300.build.build() makes it)", RuntimeWarning)
    _calls = _NotBuilt
    return _calls


def _context(stream):
    """(torch, device, raw stream) that a call goes to."""
    global _torch
    if _torch is None:
        import torch
        torch.cuda.init()
        _torch = torch
    device = _torch._C._cuda_getDevice()
    if stream is None:
        return _torch, device, _torch._C._cuda_getCurrentRawStream(device)
    return _torch, device, _stream_ptr(stream)


def _explain(name: str, t, dtype, shape, device: int):
    if not t.is_cuda:
        _refuse(f"{name}: a CUDA tensor is wanted")
    if t.get_device() != device:
        _refuse(f"{name} is on another device than the current one")
    if t.dtype is not dtype:
        _refuse(f"{name}: {t.dtype}, wanted {dtype}")
    if shape is not None and t.shape != shape:
        _refuse(f"{name}: shape {tuple(t.shape)}, wanted {tuple(shape)}")
    _refuse(f"{name} must be dense")


def _dense(name: str, t, dtype, shape, device: int) -> int:
    """Address of a dense tensor of the current device with the given type and shape (None: any)."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or (
            shape is not None and t.shape != shape):
        _explain(name, t, dtype, shape, device)
    return t.data_ptr()


def _heads(name: str, t, bf16, rows: int, heads: int, device: int):
    """Address and token stride of bf16 [rows][heads][128] whose heads lie densely."""
    shape = (rows, heads, HEAD_DIM)
    if t.dtype is not bf16 or t.get_device() != device or t.shape != shape:
        _explain(name, t, bf16, shape, device)
    stride, inner, last = t.stride()
    if last != 1 or (inner != HEAD_DIM and heads > 1):
        _refuse(f"{name}: heads must lie densely")
    return t.data_ptr(), stride if rows > 1 else heads * HEAD_DIM


# ctypes cuts an int to the argument's width without a word, so every int is checked before a call.
INT32_MIN, INT32_MAX = -2 ** 31, 2 ** 31 - 1


def _int(name: str, value) -> int:
    try:
        return operator.index(value)
    except TypeError:
        _refuse(f"{name}: an int is wanted")


def _int32(name: str, value) -> int:
    v = _int(name, value)
    if not INT32_MIN <= v <= INT32_MAX:
        _refuse(f"{name}: {v} is beyond 32 bits")
    return v


def _window(value) -> int:
    """A window beyond 32 bits holds every cache: no bound, as a negative one."""
    v = _int("window", value)
    return v if INT32_MIN <= v <= INT32_MAX else -1


def _counts(values, n: int, name: str):
    """(ctypes array, sum) of one host int per request; None stands for one each."""
    if values is None:
        return None, n
    if len(values) != n:
        _refuse(f"{name}: one per request is wanted")
    ints = [_int32(name, v) for v in values]
    if n == 0 or min(ints) < 0:
        _refuse(f"{name}: no requests, or negative")
    return (c_int32 * n)(*ints), sum(ints)


def _error_word(error, torch, device: int) -> int:
    if error.numel() < 1:
        _refuse("error: one int32 is wanted")
    return _dense("error", error, torch.int32, None, device)


def _pool(kv, torch, num_kv_heads, group, device):
    if not group:
        return _dense("kv", kv, torch.bfloat16, (kv.shape[0], num_kv_heads, 2, 64, HEAD_DIM), device)
    if group[0] not in INT4_RECORD_BYTES:
        _refuse("group_size must be 128 or 64")
    return _dense("kv", kv, torch.uint8, (kv.shape[0], num_kv_heads, INT4_RECORD_BYTES[group[0]]), device)


def _append(fn, group, kv, page_table, lens, k, v, rope, q, q_out, new_lens, interleaved, error, stream):
    st = (_calls or _marshal()).append(group[0] if group else 0, kv, page_table, lens, k, v, rope, q, q_out, new_lens,
                                    interleaved, error, stream)
    if st == 0:
        return
    if st is not None:
        _paged_check(st, "append")
    n, hkv = len(lens), _int32("kv heads", k.shape[1])
    old, _ = _counts(lens, n, "lens")
    new, rows = _counts(new_lens, n, "new_lens")
    max_pages = _int32("page_table's width", page_table.shape[1])
    torch, device, s = _context(stream)
    bf16 = torch.bfloat16
    pool = _pool(kv, torch, hkv, group, device)
    table = _dense("page_table", page_table, torch.int32, (n, max_pages), device)
    kp, ks = _heads("k", k, bf16, rows, hkv, device)
    vp, vs = _heads("v", v, bf16, rows, hkv, device)
    hq, qp, qs, qo, r, err = 0, None, 0, None, None, None
    if q is not None and q_out is not None:
        hq = _int32("query heads", q.shape[1])
        qp, qs = _heads("q", q, bf16, rows, hq, device)
        qo = _dense("q_out", q_out, bf16, (rows, hq, HEAD_DIM), device)
    elif q is not q_out:
        _refuse("q and q_out come together")
    if rope is not None:
        length, dim = (_int32("rope's shape", x) for x in rope.shape)
        r = oscar_rope(_dense("rope", rope, torch.float32, None, device), length, dim, 1 if interleaved else 0)
    if error is not None:
        err = _error_word(error, torch, device)
    if rows:
        st = fn(pool, kv.shape[0], table, max_pages, old, new, n, hq, hkv, *group, r, qp, qs, kp, ks, vp, vs, qo, err, s)
        if st:
            _paged_check(st, "append")


def bf16_append(kv, page_table, lens, k, v, rope=None, q=None, q_out=None, new_lens=None, interleaved: bool = False,
                error=None, stream=None) -> None:
    """Rotate q and k by their positions and append k and v to BF16 pages [pages][Hkv][2][64][128]: request i's
    new_lens[i] tokens (one each by default) go to positions lens[i], lens[i] + 1, ...  k, v bf16 [rows][Hkv][128] and
    q [rows][Hq][128] may be slices of one projection's output; the rotated q goes to q_out.  rope: rope_table(), or
    None for no rotation.  error: int32 [1] device word for bad page ids."""
    _append(load().oscar_bf16_append, (), kv, page_table, lens, k, v, rope, q, q_out, new_lens, interleaved, error,
            stream)


def int4_append(kv, page_table, lens, k, v, rope=None, q=None, q_out=None, new_lens=None, interleaved: bool = False,
                group_size: int = 128, error=None, stream=None) -> None:
    """bf16_append into a 4-bit pool (int4_pool), quantised per token, kv head and group of group_size channels."""
    _append(load().oscar_int4_append, (group_size,), kv, page_table, lens, k, v, rope, q, q_out, new_lens, interleaved,
            error, stream)


def int4_read(kv, page_table, starts, counts, k_out, v_out, group_size: int = 128, error=None, stream=None) -> None:
    """The values of tokens [starts[i], starts[i] + counts[i]) of each request of a 4-bit pool, into k_out and v_out
    [rows][Hkv][128], fp32 or bf16."""
    st = (_calls or _marshal()).read(group_size, kv, page_table, starts, counts, k_out, v_out, error, stream)
    if st == 0:
        return
    if st is not None:
        _paged_check(st, "read")
    n, hkv = len(starts), _int32("kv heads", kv.shape[1])
    first, _ = _counts(starts, n, "starts")
    count, rows = _counts(counts, n, "counts")
    max_pages = _int32("page_table's width", page_table.shape[1])
    torch, device, s = _context(stream)
    pool = _pool(kv, torch, hkv, (group_size,), device)
    table = _dense("page_table", page_table, torch.int32, (n, max_pages), device)
    kind = k_out.dtype
    if kind is not torch.float32 and kind is not torch.bfloat16:
        _refuse("k_out and v_out: float32 or bfloat16")
    shape = (rows, hkv, HEAD_DIM)
    ko = _dense("k_out", k_out, kind, shape, device)
    vo = _dense("v_out", v_out, kind, shape, device)
    err = None if error is None else _error_word(error, torch, device)
    if rows:
        st = load().oscar_int4_read(pool, kv.shape[0], table, max_pages, first, count, n, hkv, group_size, ko, vo,
                                    OSCAR_F32 if kind is torch.float32 else OSCAR_BF16, err, s)
        if st:
            _paged_check(st, "read")


def attention_workspace(n: int, num_q_heads: int, num_kv_heads: int, q_lens=None, stream=None):
    """Zeroed workspace for window_attention / int4_attention calls of n requests."""
    n, hq, hkv = _int32("n", n), _int32("num_q_heads", num_q_heads), _int32("num_kv_heads", num_kv_heads)
    rows, _ = _counts(q_lens, n, "q_lens")
    torch, device, s = _context(stream)
    need = load().oscar_attention_workspace_bytes(n, rows, hq, hkv)
    if need == 0:
        _refuse("arguments outside the supported limits")
    with torch.cuda.stream(None if stream is None else torch.cuda.ExternalStream(s, device)):
        return new_workspace(need)


def _attention(fn, group, kv, page_table, lens, q, out, hkv, window, sinks, q_lens, scale, lse, workspace, error,
               stream):
    st = (_calls or _marshal()).attend(group[0] if group else 0, kv, page_table, lens, q, out, hkv, window, sinks, q_lens,
                                    scale, lse, workspace, error, stream)
    if st == 0:
        return workspace
    if st is not None and load().oscar_paged_last_error() != b"workspace too small":
        _paged_check(st, "attention")
    n, hq, hkv = len(lens), _int32("query heads", q.shape[1]), _int32("num_kv_heads", hkv)
    window, sinks = _window(window), _int32("sinks", sinks)
    total, _ = _counts(lens, n, "lens")
    new, rows = _counts(q_lens, n, "q_lens")
    max_pages = _int32("page_table's width", page_table.shape[1])
    torch, device, s = _context(stream)
    kind, f32 = out.dtype, torch.float32
    pool = _pool(kv, torch, hkv, group, device)
    table = _dense("page_table", page_table, torch.int32, (n, max_pages), device)
    qp, qs = _heads("q", q, torch.bfloat16, rows, hq, device)
    if kind is not f32 and kind is not torch.bfloat16:
        _refuse("out: float32 or bfloat16")
    op = _dense("out", out, kind, (rows, hq, HEAD_DIM), device)
    lp = None if lse is None else _dense("lse", lse, f32, (rows, hq), device)
    err = None if error is None else _error_word(error, torch, device)
    if workspace is None:
        workspace = attention_workspace(n, hq, hkv, q_lens, stream)
    while rows:
        st = fn(pool, kv.shape[0], table, max_pages, total, new, n, hq, hkv, *group, window, sinks, scale, qp, qs, op,
                OSCAR_F32 if kind is f32 else OSCAR_BF16, lp, err,
                _dense("workspace", workspace, torch.uint8, None, device), workspace.numel(), s)
        if not st:
            break
        if load().oscar_paged_last_error() != b"workspace too small":
            _paged_check(st, "attention")
        workspace = attention_workspace(n, hq, hkv, q_lens, stream)
    return workspace


def window_attention(kv, page_table, lens, q, out, num_kv_heads: int, window: int = -1, sinks: int = 0, q_lens=None,
                     scale: float = 0.0, lse=None, workspace=None, error=None, stream=None):
    """Attention of the last q_lens[i] positions (one each by default) of every request over BF16 pages: the query at
    position p sees the tokens t <= p with t < sinks or t > p - window (window < 0, or beyond 32 bits: no bound).  q
    bf16 [rows][Hq][128] (rows may be strided), out [rows][Hq][128] fp32 or bf16, lse fp32 [rows][Hq] or None.  Returns
    the workspace to pass to the next call: a new one where none is given or it is too small (attention_workspace()
    makes one)."""
    return _attention(load().oscar_window_attention, (), kv, page_table, lens, q, out, num_kv_heads, window, sinks,
                      q_lens, scale, lse, workspace, error, stream)


def int4_attention(kv, page_table, lens, q, out, num_kv_heads: int, window: int = -1, sinks: int = 0, q_lens=None,
                   group_size: int = 128, scale: float = 0.0, lse=None, workspace=None, error=None, stream=None):
    """window_attention over a 4-bit pool, for at most 16 / (Hq / Hkv) query tokens a request."""
    return _attention(load().oscar_int4_attention, (group_size,), kv, page_table, lens, q, out, num_kv_heads, window,
                      sinks, q_lens, scale, lse, workspace, error, stream)
