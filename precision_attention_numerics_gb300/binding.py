"""ctypes binding of libattnq (include/attnq.h).  Argument marshalling only.

Tensor arguments are torch tensors on the current CUDA device (their data
pointers are passed through); `stream` defaults to torch's current stream.
Every function raises AttnqError on a non-OK status.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from dataclasses import dataclass
from typing import Optional

import numpy as np

ATTNQ_ROTATE = 1
ATTNQ_CENTER_K = 2
ATTNQ_VT_LAYOUT = 4
ATTNQ_TILE_SCALES = 8
ATTNQ_I8QK = 16
ATTNQ_SCALE_TILE = 128
ATTNQ_F32 = 0
ATTNQ_BF16 = 1
ATTNQ_KV_FORWARD = 0
ATTNQ_KV_REVERSE = 1

STATUS = {0: "ATTNQ_OK", 1: "ATTNQ_EINVAL", 2: "ATTNQ_EUNSUPPORTED", 3: "ATTNQ_ECUDA", 4: "ATTNQ_ENONFINITE",
          5: "ATTNQ_ETIMEOUT", 6: "ATTNQ_EPAGE"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libattnq.so")
_lib = None


class AttnqError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


class _Desc(C.Structure):
    _fields_ = [("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("N", C.c_int32), ("d", C.c_int32),
                ("in_dtype", C.c_int32), ("flags", C.c_uint32), ("signs", C.c_void_p), ("stat_len", C.c_int32)]


class _Scales(C.Structure):
    _fields_ = [("q_descale", C.c_void_p), ("k_descale", C.c_void_p), ("v_descale", C.c_void_p),
                ("k_mean", C.c_void_p)]


@dataclass
class AttnqDesc:
    """Mirror of attnq_desc; `signs` is a device int8 tensor of d values or None;
    `stat_len` = P takes the mean key and the per-(batch, head) scales over the
    first P tokens (0: all N)."""
    B: int
    Hq: int
    Hkv: int
    N: int
    d: int
    in_dtype: int = ATTNQ_BF16
    flags: int = ATTNQ_VT_LAYOUT
    signs: Optional[object] = None
    stat_len: int = 0

    def _c(self) -> _Desc:
        return _Desc(self.B, self.Hq, self.Hkv, self.N, self.d, self.in_dtype, self.flags,
                     None if self.signs is None else self.signs.data_ptr(), self.stat_len)


@dataclass
class AttnqScales:
    """Mirror of attnq_scales (device fp32 tensors; k_mean optional)."""
    q_descale: object
    k_descale: object
    v_descale: object
    k_mean: Optional[object] = None

    def _c(self) -> _Scales:
        return _Scales(self.q_descale.data_ptr(), self.k_descale.data_ptr(), self.v_descale.data_ptr(),
                       None if self.k_mean is None else self.k_mean.data_ptr())


class _Kv4Cache(C.Structure):
    _fields_ = [("num_pages", C.c_int32), ("page_tokens", C.c_int32), ("Hkv", C.c_int32), ("d", C.c_int32),
                ("flags", C.c_uint32), ("signs", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("pages", C.c_void_p)]


class _Kv4Seqs(C.Structure):
    _fields_ = [("B", C.c_int32), ("max_pages", C.c_int32), ("table", C.c_void_p), ("lens", C.c_void_p),
                ("new_lens", C.c_void_p)]


class _Rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("dtype", C.c_int32), ("stride_b", C.c_int64), ("stride_h", C.c_int64),
                ("stride_t", C.c_int64)]


# The same layouts as bytes: a call packs its three to five structs in a third of the time that
# ctypes takes to build them (their sum is a fifth of a small call's host time).
_pack_kv4_cache = struct.Struct("=iiiiI4xQQQQ").pack
_pack_kv4_seqs = struct.Struct("=iiQQQ").pack
_pack_rows = struct.Struct("=Qi4xqqq").pack


@dataclass
class AttnqKv4Cache:
    """Mirror of attnq_kv4_cache; `signs` is a device int8 tensor of d values or
    None, `k_scale` and `v_scale` device fp32 [Hkv] or None, `pages` a device
    uint8 tensor of attnq_kv4_cache_bytes(cache) bytes (alloc_kv4_cache makes one)."""
    num_pages: int
    page_tokens: int
    Hkv: int
    d: int
    flags: int = 0
    signs: Optional[object] = None
    k_scale: Optional[object] = None
    v_scale: Optional[object] = None
    pages: Optional[object] = None

    def _c(self) -> _Kv4Cache:
        return _Kv4Cache(self.num_pages, self.page_tokens, self.Hkv, self.d, self.flags,
                         *(None if t is None else t.data_ptr()
                           for t in (self.signs, self.k_scale, self.v_scale, self.pages)))


@dataclass
class AttnqKv4Seqs:
    """Mirror of attnq_kv4_seqs: device int32 `table` [B, max_pages], `lens` [B]
    (tokens of each sequence, the call's own among them) and optional
    `new_lens` [B] (rows of the call that belong to each sequence)."""
    table: object
    lens: object
    new_lens: Optional[object] = None

    def _c(self) -> _Kv4Seqs:
        return _Kv4Seqs(self.table.shape[0], self.table.shape[1], self.table.data_ptr(), self.lens.data_ptr(),
                        None if self.new_lens is None else self.new_lens.data_ptr())


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libattnq.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(python -m precision_attention_numerics_gb300._build)")
    L = C.CDLL(_LIB_PATH)
    P, i32, u32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_uint32, C.c_int64, C.c_float, C.c_size_t
    L.attnq_version.restype = i32
    L.attnq_status_string.restype = C.c_char_p
    L.attnq_status_string.argtypes = [i32]
    L.attnq_vt_ld.restype = i64
    L.attnq_vt_ld.argtypes = [i32]
    L.attnq_scale_tiles.restype = i32
    L.attnq_scale_tiles.argtypes = [i32]
    L.attnq_hadamard_signs.restype = i32
    L.attnq_hadamard_signs.argtypes = [C.c_uint64, i32, P]
    L.attnq_prepare_workspace.restype = sz
    L.attnq_prepare_workspace.argtypes = [P]
    L.attnq_prepare.restype = i32
    L.attnq_prepare.argtypes = [P, P, P, P, P, P, P, P, P, sz, P]
    L.attnq_prepare_static.restype = i32
    L.attnq_prepare_static.argtypes = [P, P, P, P, P, P, P, P, P]
    L.attnq_fwd.restype = i32
    L.attnq_fwd.argtypes = [P, P, P, P, P, f32, i32, i32, i32, P, i32, P, i32, P]
    L.attnq_fwd_ponly.restype = i32
    L.attnq_fwd_ponly.argtypes = [P, P, P, P, f32, i32, i32, i32, P, P, i32, P]
    L.attnq_err.restype = i32
    L.attnq_err.argtypes = [P, P, i32, P, P, P]
    L.attnq_device_status.restype = i32
    L.attnq_device_status.argtypes = [P]
    L.attnq_set_wait_limit_ns.restype = C.c_uint64
    L.attnq_set_wait_limit_ns.argtypes = [C.c_uint64]
    L.attnq_ref_attention.restype = i32
    L.attnq_ref_attention.argtypes = [P, P, P, P, i32, P, P]
    L.attnq_harm_workspace.restype = sz
    L.attnq_harm_workspace.argtypes = [P]
    L.attnq_harm_report.restype = i32
    L.attnq_harm_report.argtypes = [P, P, P, P, f32, i32, i32, P, sz, P, P]
    L.attnq_host_pipeline_workspace.restype = sz
    L.attnq_host_pipeline_workspace.argtypes = [P, i32]
    L.attnq_attention_host.restype = i32
    L.attnq_attention_host.argtypes = [P, i32, P, P, P, f32, i32, i32, i32, P, i32, P, sz, P, P, P]
    L.attnq_kv4_cache_bytes.restype = sz
    L.attnq_kv4_cache_bytes.argtypes = [P]
    L.attnq_kv4_append.restype = i32
    L.attnq_kv4_append.argtypes = [P, P, i32, P, P, P, P]
    L.attnq_kv4_read.restype = i32
    L.attnq_kv4_read.argtypes = [P, P, i32, P, P, P]
    L.attnq_kv4_attn_workspace.restype = sz
    L.attnq_kv4_attn_workspace.argtypes = [P, i32, i32, i32, i32]
    L.attnq_kv4_attn.restype = i32
    L.attnq_kv4_attn.argtypes = [P, P, i32, i32, P, P, f32, i32, P, P, P, P, sz, P]
    L.attnq_kv4_evict_workspace.restype = sz
    L.attnq_kv4_evict_workspace.argtypes = [P, i32, i32, i32]
    L.attnq_kv4_evict.restype = i32
    L.attnq_kv4_evict.argtypes = [P, P, P, i32, i32, i32, P, i32, P, P, P, P, sz, P]
    _lib = L
    return L


def exported_symbols() -> list[str]:
    """Names declared in include/attnq.h (for the ABI test)."""
    import re
    hdr = os.path.join(os.path.dirname(_HERE), "include", "attnq.h")
    text = open(hdr).read()
    return sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(attnq_\w+)\s*\(", text, flags=re.M)))


def _stream(stream):
    if stream is not None:
        return C.c_void_p(int(stream))
    import torch
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _check(code: int, what: str):
    if code != 0:
        raise AttnqError(code, what)


def attnq_version() -> int:
    return int(load_library().attnq_version())


def attnq_status_string(code: int) -> str:
    return load_library().attnq_status_string(code).decode()


def attnq_vt_ld(N: int) -> int:
    return int(load_library().attnq_vt_ld(N))


def attnq_scale_tiles(N: int) -> int:
    return int(load_library().attnq_scale_tiles(N))


def attnq_hadamard_signs(seed: int, d: int) -> np.ndarray:
    out = np.empty(d, dtype=np.int8)
    _check(load_library().attnq_hadamard_signs(C.c_uint64(seed), d, out.ctypes.data_as(C.c_void_p)),
           "attnq_hadamard_signs")
    return out


def attnq_prepare_workspace(desc: AttnqDesc) -> int:
    d = desc._c()
    return int(load_library().attnq_prepare_workspace(C.byref(d)))


def attnq_prepare(desc: AttnqDesc, Q, K, V, q8, k8, v8, scales: AttnqScales, workspace, stream=None) -> None:
    d, s = desc._c(), scales._c()
    nbytes = workspace.numel() * workspace.element_size()
    _check(load_library().attnq_prepare(C.byref(d), _ptr(Q), _ptr(K), _ptr(V), _ptr(q8), _ptr(k8), _ptr(v8),
                                        C.byref(s), _ptr(workspace), nbytes, _stream(stream)), "attnq_prepare")


def attnq_prepare_static(desc: AttnqDesc, Q, K, V, q8, k8, v8, scales: AttnqScales, stream=None) -> None:
    """attnq_prepare with the library's fixed scratch array instead of a workspace
    (for callers that cannot allocate; calls must not overlap on the GPU)."""
    d, s = desc._c(), scales._c()
    _check(load_library().attnq_prepare_static(C.byref(d), _ptr(Q), _ptr(K), _ptr(V), _ptr(q8), _ptr(k8), _ptr(v8),
                                               C.byref(s), _stream(stream)), "attnq_prepare_static")


ATTNQ_STATIC_SCRATCH_BYTES = 4 << 20


def attnq_fwd(desc: AttnqDesc, q8, k8, v8, scales: AttnqScales, S: float, kv_order: int, causal: bool,
              kv_tile: int, O, underflow=None, k_sink: int = 4, stream=None) -> None:
    import torch
    d, s = desc._c(), scales._c()
    out_dtype = ATTNQ_BF16 if O.dtype == torch.bfloat16 else ATTNQ_F32
    _check(load_library().attnq_fwd(C.byref(d), _ptr(q8), _ptr(k8), _ptr(v8), C.byref(s), float(S), int(kv_order),
                                    int(bool(causal)), int(kv_tile), _ptr(O), out_dtype, _ptr(underflow),
                                    int(k_sink), _stream(stream)), "attnq_fwd")


def attnq_fwd_ponly(desc: AttnqDesc, Q, K, V, S: float, kv_order: int, causal: bool, kv_tile: int, O,
                    underflow=None, k_sink: int = 4, stream=None) -> None:
    d = desc._c()
    _check(load_library().attnq_fwd_ponly(C.byref(d), _ptr(Q), _ptr(K), _ptr(V), float(S), int(kv_order),
                                          int(bool(causal)), int(kv_tile), _ptr(O), _ptr(underflow), int(k_sink),
                                          _stream(stream)), "attnq_fwd_ponly")


def attnq_err(desc: AttnqDesc, O, O_ref, err_out, stream=None) -> None:
    import torch
    d = desc._c()
    o_dtype = ATTNQ_BF16 if O.dtype == torch.bfloat16 else ATTNQ_F32
    _check(load_library().attnq_err(C.byref(d), _ptr(O), o_dtype, _ptr(O_ref), _ptr(err_out), _stream(stream)),
           "attnq_err")


def attnq_device_status(stream=None) -> int:
    """Synchronise and return (and clear) the device status code (0 = OK)."""
    return int(load_library().attnq_device_status(_stream(stream)))


def attnq_ref_attention(desc: AttnqDesc, Q, K, V, causal: bool, O_ref, stream=None) -> None:
    """FP64 reference attention of the original inputs into O_ref (fp64 [B,Hq,N,d])."""
    d = desc._c()
    _check(load_library().attnq_ref_attention(C.byref(d), _ptr(Q), _ptr(K), _ptr(V), int(bool(causal)),
                                              _ptr(O_ref), _stream(stream)), "attnq_ref_attention")


def attnq_harm_workspace(desc: AttnqDesc) -> int:
    d = desc._c()
    return int(load_library().attnq_harm_workspace(C.byref(d)))


def attnq_harm_report(desc: AttnqDesc, Q, K, V, S: float, kv_order: int, kv_tile: int, workspace, err_out,
                      stream=None) -> None:
    """Per-head errors of the four conditions into err_out (fp64 [4, B*Hq])."""
    d = desc._c()
    _check(load_library().attnq_harm_report(C.byref(d), _ptr(Q), _ptr(K), _ptr(V), float(S), int(kv_order),
                                            int(kv_tile), _ptr(workspace), workspace.numel(), _ptr(err_out),
                                            _stream(stream)), "attnq_harm_report")


def attnq_set_wait_limit_ns(ns: int) -> int:
    """Set the limit of every wait inside the kernels (nanoseconds); returns the previous one."""
    return int(load_library().attnq_set_wait_limit_ns(int(ns)))


def attnq_host_pipeline_workspace(desc: AttnqDesc, out_dtype: int) -> int:
    d = desc._c()
    return int(load_library().attnq_host_pipeline_workspace(C.byref(d), int(out_dtype)))


def attnq_attention_host(desc: AttnqDesc, Q_host, K_host, V_host, S: float, kv_order: int, causal: bool,
                         kv_tile: int, O_host, out_dtype: int, workspace, compute, copy_in, copy_out) -> None:
    """Prepare + attention over n steps whose inputs and outputs live in host
    memory (lists of pinned CPU tensors of equal length); see include/attnq.h.
    `compute`, `copy_in`, `copy_out`: three torch.cuda.Stream objects."""
    n = len(Q_host)
    if not (len(K_host) == len(V_host) == len(O_host) == n):
        raise ValueError("Q_host, K_host, V_host and O_host must have one entry per step")
    arr = C.c_void_p * max(n, 1)
    qa, ka, va, oa = (arr(*[t.data_ptr() for t in ts]) for ts in (Q_host, K_host, V_host, O_host))
    d = desc._c()
    _check(load_library().attnq_attention_host(
        C.byref(d), n, qa, ka, va, float(S), int(kv_order), int(bool(causal)), int(kv_tile), oa, int(out_dtype),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(compute.cuda_stream),
        _stream(copy_in.cuda_stream), _stream(copy_out.cuda_stream)), "attnq_attention_host")


def _refuse(what: str):
    raise AttnqError(1, what)


def _int32(*values) -> bool:
    """Whether a call's int32 arguments can hold these (ctypes cuts longer ones off in silence)."""
    return -(1 << 31) <= min(values) and max(values) < 1 << 31


def _kv4_sizes(cache: AttnqKv4Cache) -> Optional[_Kv4Cache]:
    """The cache's struct for the functions that ask for bytes; None (0 bytes) where its sizes do not fit."""
    return cache._c() if _int32(cache.num_pages, cache.page_tokens, cache.Hkv, cache.d) else None


def _kv4_ptr(t, what: str, name: str, dtype, dev: int, shape=None) -> int:
    """Address of a contiguous tensor of device `dev`, of the given type and shape."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (shape is not None and
                                                                                  t.shape != shape):
        _refuse(f"{what}: {name} must be contiguous {dtype} on the current CUDA device"
                + ("" if shape is None else f" of shape {tuple(shape)}"))
    return t.data_ptr()


def _kv4_structs(what: str, cache: AttnqKv4Cache, seqs: AttnqKv4Seqs, dev: int):
    """Checked C structs of a call's cache and sequences (as bytes), and B and max_pages."""
    import torch
    Hkv, d = cache.Hkv, cache.d
    pages, signs, gk, gv = cache.pages, cache.signs, cache.k_scale, cache.v_scale
    if pages is None or pages.numel() < cache.num_pages * cache.page_tokens * Hkv * (d + d // 8):
        _refuse(f"{what}: the cache has fewer than attnq_kv4_cache_bytes(cache) bytes of pages")
    table, new_lens = seqs.table, seqs.new_lens
    if table.dim() != 2:
        _refuse(f"{what}: table must be [B, max_pages]")
    B, max_pages = table.shape
    try:
        c = _pack_kv4_cache(cache.num_pages, cache.page_tokens, Hkv, d, cache.flags,
                            0 if signs is None else _kv4_ptr(signs, what, "signs", torch.int8, dev, (d,)),
                            0 if gk is None else _kv4_ptr(gk, what, "k_scale", torch.float32, dev, (Hkv,)),
                            0 if gv is None else _kv4_ptr(gv, what, "v_scale", torch.float32, dev, (Hkv,)),
                            _kv4_ptr(pages, what, "pages", torch.uint8, dev))
        s = _pack_kv4_seqs(B, max_pages, _kv4_ptr(table, what, "table", torch.int32, dev),
                           _kv4_ptr(seqs.lens, what, "lens", torch.int32, dev, (B,)),
                           0 if new_lens is None else _kv4_ptr(new_lens, what, "new_lens", torch.int32, dev, (B,)))
    except struct.error:  # a size that 32 bits do not hold
        _refuse(f"{what}: a size of the cache or the table")
    return c, s, B, max_pages


def _kv4_rows(t, what: str, name: str, dev: int, B: int, H: int, T: int, d: int) -> bytes:
    """attnq_rows of a [B, H, T, d] tensor (any strides, d contiguous)."""
    import torch
    dt, stride = t.dtype, t.stride()
    if dt is torch.bfloat16:
        code = ATTNQ_BF16
    elif dt is torch.float32:
        code = ATTNQ_F32
    else:
        _refuse(f"{what}: {name} must be bfloat16 or float32")
    if t.get_device() != dev or t.shape != (B, H, T, d) or stride[3] != 1 or H >> 31 or T >> 31:
        _refuse(f"{what}: {name} must be [{B}, {H}, {T}, {d}] on the current CUDA device, its last axis contiguous")
    return _pack_rows(t.data_ptr(), code, stride[0], stride[1], stride[2])


def _kv4_device() -> int:
    import torch
    return torch.cuda.current_device()


def _kv4_stream(stream, dev: int):
    """`stream`, or torch's current one (its handle alone: building a Stream object takes 3 us of a call's 15)."""
    if stream is not None:
        return int(stream)
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else torch.cuda.current_stream().cuda_stream


def attnq_kv4_cache_bytes(cache: AttnqKv4Cache) -> int:
    c = _kv4_sizes(cache)
    return int(load_library().attnq_kv4_cache_bytes(C.byref(c))) if c is not None else 0


def _kv4_rows_call(fn, what: str, cache, seqs, K, V, names, k_mean, stream) -> None:
    import torch
    dev = _kv4_device()
    c, s, B, _ = _kv4_structs(what, cache, seqs, dev)
    if K.dim() != 4:
        _refuse(f"{what}: {names[0]} must be [B, Hkv, T, d]")
    T = K.shape[2]
    k = _kv4_rows(K, what, names[0], dev, B, cache.Hkv, T, cache.d)
    v = _kv4_rows(V, what, names[1], dev, B, cache.Hkv, T, cache.d)
    mean = ()
    if what == "attnq_kv4_append":
        mean = (None if k_mean is None else
                _kv4_ptr(k_mean, what, "k_mean", torch.float32, dev, (B, cache.Hkv, cache.d)),)
    _check(fn(c, s, T, k, v, *mean, _kv4_stream(stream, dev)), what)


def attnq_kv4_append(cache: AttnqKv4Cache, seqs: AttnqKv4Seqs, K, V, k_mean=None, stream=None) -> None:
    """Quantise the rows K, V [B, Hkv, T, d] (bf16 or fp32, any strides with d
    contiguous) into the cache; see include/attnq.h."""
    _kv4_rows_call(load_library().attnq_kv4_append, "attnq_kv4_append", cache, seqs, K, V, ("K", "V"), k_mean, stream)


def attnq_kv4_read(cache: AttnqKv4Cache, seqs: AttnqKv4Seqs, K_out, V_out, stream=None) -> None:
    """The values held for the rows that attnq_kv4_append writes, into K_out and V_out [B, Hkv, T, d]."""
    _kv4_rows_call(load_library().attnq_kv4_read, "attnq_kv4_read", cache, seqs, K_out, V_out, ("K_out", "V_out"), None,
                   stream)


def attnq_kv4_attn_workspace(cache: AttnqKv4Cache, B: int, max_pages: int, Hq: int, T: int) -> int:
    c, B, max_pages, Hq, T = _kv4_sizes(cache), int(B), int(max_pages), int(Hq), int(T)
    if c is None or not _int32(B, max_pages, Hq, T):
        return 0
    return int(load_library().attnq_kv4_attn_workspace(C.byref(c), B, max_pages, Hq, T))


def attnq_kv4_attn(cache: AttnqKv4Cache, seqs: AttnqKv4Seqs, Q, O, causal: bool, workspace, scale=None, lse=None,
                   acc_in=None, acc_out=None, stream=None) -> None:
    """Attention of the rows Q [B, Hq, T, d] over the cache into O; `scale` is
    1/sqrt(d) unless given; optional `lse` [B, Hq, T] and accumulated weights
    `acc_out` [B, Hkv, max_pages * page_tokens] (= `acc_in`, or 0, plus this call's)."""
    import torch
    what, dev = "attnq_kv4_attn", _kv4_device()
    c, s, B, max_pages = _kv4_structs(what, cache, seqs, dev)
    if Q.dim() != 4:
        _refuse(f"{what}: Q must be [B, Hq, T, d]")
    Hq, T = Q.shape[1], Q.shape[2]
    q = _kv4_rows(Q, what, "Q", dev, B, Hq, T, cache.d)
    o = _kv4_rows(O, what, "O", dev, B, Hq, T, cache.d)
    f32 = torch.float32
    p_lse = p_in = p_out = None
    if lse is not None:
        p_lse = _kv4_ptr(lse, what, "lse", f32, dev, (B, Hq, T))
    if acc_out is not None:
        p_out = _kv4_ptr(acc_out, what, "acc_out", f32, dev, (B, cache.Hkv, max_pages * cache.page_tokens))
    if acc_in is not None:
        p_in = _kv4_ptr(acc_in, what, "acc_in", f32, dev, (B, cache.Hkv, max_pages * cache.page_tokens))
    _check(load_library().attnq_kv4_attn(
        c, s, T, Hq, q, o, cache.d ** -0.5 if scale is None else float(scale),
        1 if causal else 0, p_lse, p_in, p_out, _kv4_ptr(workspace, what, "workspace", workspace.dtype, dev),
        workspace.nbytes, _kv4_stream(stream, dev)), what)


def attnq_kv4_evict_workspace(cache: AttnqKv4Cache, B: int, max_pages: int, budget: int) -> int:
    c, B, max_pages, budget = _kv4_sizes(cache), int(B), int(max_pages), int(budget)
    if c is None or not _int32(B, max_pages, budget):
        return 0
    return int(load_library().attnq_kv4_evict_workspace(C.byref(c), B, max_pages, budget))


def attnq_kv4_evict(cache: AttnqKv4Cache, seqs: AttnqKv4Seqs, acc, budget: int, n_sink: int, n_recent: int,
                    dst_table, new_lens, kept, acc_out, workspace, stream=None) -> None:
    """Keep at most `budget` tokens per KV head (the first n_sink, the last
    n_recent, and the largest accumulated weights `acc` between), moved to the pages
    of `dst_table` [B, dst_pages]; writes `new_lens` [B], `kept` [B, Hkv, budget]
    and, unless None, `acc_out` [B, Hkv, dst_pages * page_tokens]."""
    import torch
    what, dev = "attnq_kv4_evict", _kv4_device()
    c, s, B, max_pages = _kv4_structs(what, cache, seqs, dev)
    Hkv, page, f32, i32, budget = cache.Hkv, cache.page_tokens, torch.float32, torch.int32, int(budget)
    if dst_table.dim() != 2 or dst_table.shape[0] != B:
        _refuse(f"{what}: dst_table must be [B, dst_pages]")
    dst_pages, n_sink, n_recent = dst_table.shape[1], int(n_sink), int(n_recent)
    if not _int32(budget, n_sink, n_recent, dst_pages):
        _refuse(f"{what}: budget, n_sink, n_recent or dst_pages")
    _check(load_library().attnq_kv4_evict(
        c, s, _kv4_ptr(acc, what, "acc", f32, dev, (B, Hkv, max_pages * page)), budget,
        n_sink, n_recent, _kv4_ptr(dst_table, what, "dst_table", i32, dev), dst_pages,
        _kv4_ptr(new_lens, what, "new_lens", i32, dev, (B,)), _kv4_ptr(kept, what, "kept", i32, dev, (B, Hkv, budget)),
        None if acc_out is None else _kv4_ptr(acc_out, what, "acc_out", f32, dev, (B, Hkv, dst_pages * page)),
        _kv4_ptr(workspace, what, "workspace", workspace.dtype, dev), workspace.nbytes, _kv4_stream(stream, dev)), what)
