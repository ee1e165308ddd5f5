"""CacheGen-style KV-cache codec for AMD MI355X: Python binding of libkvc.so.

The functions named kvc_* mirror the C ABI in include/kvc.h one to one and
only marshal arguments (torch tensors -> device pointers, the caller's HIP
stream).  Every step of the codec runs in the HIP kernels of libkvc.so; there
is no CPU path.  `encode` / `decode` chain those calls for convenience.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvc.so")

KVC_OK, KVC_ERR_ARG, KVC_ERR_CAPACITY, KVC_ERR_HIP = 0, -1, -2, -3
KVC_DEV_NONFINITE, KVC_DEV_CORRUPT, KVC_DEV_PAYLOAD_OVERFLOW = 1, 2, 4
KVC_DEV_BAD_CDF, KVC_DEV_BAD_CONTAINER, KVC_DEV_BAD_SYMBOL = 8, 16, 32
KVC_DEV_BAD_INDEX = 64
KVC_F16, KVC_F32, KVC_BF16 = 0, 1, 2

EXPORTED = (
    "kvc_version", "kvc_status_string", "kvc_alphabet", "kvc_n_chunks", "kvc_n_slabs",
    "kvc_n_streams", "kvc_cdf_bytes", "kvc_scratch_bytes", "kvc_max_payload_bytes",
    "kvc_quantize", "kvc_cdf", "kvc_encode", "kvc_decode", "kvc_dequantize",
    "kvc_container_bytes", "kvc_container_payload_offset", "kvc_serialize", "kvc_deserialize",
    "kvc_int8_quantize", "kvc_int8_dequantize", "kvc_serialize_chunk", "kvc_quantize_levels",
    "kvc_decode_lanes", "kvc_delta_forward", "kvc_delta_inverse", "kvc_encode_noalloc",
    "kvc_stream_work_bytes", "kvc_stream_encode",
    "kvc_kv4_codes_bytes", "kvc_kv4_params_bytes", "kvc_kv4_append", "kvc_kv4_read",
    "kvc_kv4_work_bytes", "kvc_kv4_attention",
)
KVC_NOALLOC_SCRATCH_BYTES = 64 << 20


class KvcDesc(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int32),
        ("n_channels", ctypes.c_int32),
        ("n_tokens", ctypes.c_int64),
        ("chunk_tokens", ctypes.c_int32),
        ("cdf_chunks", ctypes.c_int32),
        ("bins", ctypes.POINTER(ctypes.c_int32)),
    ]


class KvcKv4Desc(ctypes.Structure):
    _fields_ = [
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("n_pages", ctypes.c_int64),
    ]


class KvcKv4Attn(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("kv_len", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
        ("n_q", ctypes.c_int64),
        ("n_seqs", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("max_q", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
        ("softcap", ctypes.c_float), ("scale", ctypes.c_float),
        ("work", ctypes.c_void_p), ("work_bytes", ctypes.c_int64),
    ]


# void on_chunk(void *user, int64_t chunk, int32_t level, const uint8_t *container, int64_t n_bytes)
CHUNK_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                            ctypes.c_int64)


class KvcError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = _load().kvc_status_string(status).decode() if _lib else str(status)
        super().__init__(f"{fn} failed: {msg} ({status})")


_lib = None


def _load():
    """Load libkvc.so; fail loudly when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m entropy_coding_02_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D = ctypes.POINTER(KvcDesc)
        lib.kvc_version.restype = ctypes.c_int
        lib.kvc_status_string.restype = ctypes.c_char_p
        lib.kvc_status_string.argtypes = [ctypes.c_int]
        lib.kvc_alphabet.restype = I32
        lib.kvc_decode_lanes.restype = I32
        lib.kvc_decode_lanes.argtypes = [D]
        lib.kvc_delta_forward.restype = ctypes.c_int
        lib.kvc_delta_forward.argtypes = [D, I32, P, P, P, P]
        lib.kvc_delta_inverse.restype = ctypes.c_int
        lib.kvc_delta_inverse.argtypes = [D, I32, P, P]
        for n in ("kvc_n_chunks", "kvc_n_slabs", "kvc_n_streams", "kvc_cdf_bytes",
                  "kvc_scratch_bytes", "kvc_max_payload_bytes"):
            getattr(lib, n).restype = I64
        for n in ("kvc_alphabet", "kvc_n_chunks", "kvc_n_slabs", "kvc_n_streams", "kvc_cdf_bytes",
                  "kvc_scratch_bytes", "kvc_max_payload_bytes"):
            getattr(lib, n).argtypes = [D]
        lib.kvc_quantize.restype = ctypes.c_int
        lib.kvc_quantize.argtypes = [D, P, P, P, P, P, P]
        lib.kvc_cdf.restype = ctypes.c_int
        lib.kvc_cdf.argtypes = [D, P, P, P, P]
        lib.kvc_encode.restype = ctypes.c_int
        lib.kvc_encode.argtypes = [D, P, P, P, I64, P, P, P, I64, P, P]
        lib.kvc_encode_noalloc.restype = ctypes.c_int
        lib.kvc_encode_noalloc.argtypes = [D, P, P, P, P, P, I64, P, P]
        lib.kvc_decode.restype = ctypes.c_int
        lib.kvc_decode.argtypes = [D, P, I64, P, P, P, P, P, P, I32, P, P]
        lib.kvc_dequantize.restype = ctypes.c_int
        lib.kvc_dequantize.argtypes = [D, P, P, P, I32, P]
        lib.kvc_container_bytes.restype = I64
        lib.kvc_container_bytes.argtypes = [D, I64]
        lib.kvc_container_payload_offset.restype = I64
        lib.kvc_container_payload_offset.argtypes = [D]
        lib.kvc_serialize.restype = ctypes.c_int
        lib.kvc_serialize.argtypes = [D, P, P, P, P, P, P, I64, P, P]
        lib.kvc_deserialize.restype = ctypes.c_int
        lib.kvc_deserialize.argtypes = [D, P, I64, P, P, P, P, P, P]
        lib.kvc_quantize_levels.restype = ctypes.c_int
        lib.kvc_quantize_levels.argtypes = [D, I32, P, P, P, P, P, P]
        lib.kvc_serialize_chunk.restype = ctypes.c_int
        lib.kvc_serialize_chunk.argtypes = [D, I64, P, P, P, P, P, P, I64, P, P]
        lib.kvc_int8_quantize.restype = ctypes.c_int
        lib.kvc_int8_quantize.argtypes = [D, I32, P, P, P, P, P, P]
        lib.kvc_int8_dequantize.restype = ctypes.c_int
        lib.kvc_int8_dequantize.argtypes = [D, I32, P, P, P, P, I32, P]
        lib.kvc_stream_work_bytes.restype = I64
        lib.kvc_stream_work_bytes.argtypes = [D, I32, I32]
        lib.kvc_stream_encode.restype = ctypes.c_int
        lib.kvc_stream_encode.argtypes = [D, I32, P, P, P, P, I32, P, I64, P, I64, P, P, P, P,
                                          CHUNK_FN, P]
        K = ctypes.POINTER(KvcKv4Desc)
        lib.kvc_kv4_codes_bytes.restype = I64
        lib.kvc_kv4_codes_bytes.argtypes = [K]
        lib.kvc_kv4_params_bytes.restype = I64
        lib.kvc_kv4_params_bytes.argtypes = [K]
        lib.kvc_kv4_append.restype = ctypes.c_int
        lib.kvc_kv4_append.argtypes = [K, P, P, I64, I64, I64, I64, I64, I32, P, P, P, P, P]
        lib.kvc_kv4_read.restype = ctypes.c_int
        lib.kvc_kv4_read.argtypes = [K, P, P, P, I64, P, P, I64, I64, I64, I64, I32, P, P]
        lib.kvc_kv4_work_bytes.restype = I64
        lib.kvc_kv4_work_bytes.argtypes = [K, I64, I32, I32, I32, I32]
        lib.kvc_kv4_attention.restype = ctypes.c_int
        lib.kvc_kv4_attention.argtypes = [K, P, P, P, P, P]  # the kvc_kv4_attn as bytes or a reference
        _lib = lib
    return _lib


def lib():
    return _load()


class Desc:
    """A kvc_desc plus the host bins array it points to."""

    def __init__(self, n_layers: int, n_channels: int, n_tokens: int, bins,
                 chunk_tokens: int = 256, cdf_chunks: int = 0):
        """cdf_chunks: chunks sharing one CDF table (0 or 1: a table per chunk)."""
        self.bins = np.ascontiguousarray(np.asarray(bins, dtype=np.int32).reshape(n_layers, 2))
        self.c = KvcDesc(n_layers, n_channels, n_tokens, chunk_tokens, cdf_chunks,
                         self.bins.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
        self.n_layers, self.n_channels, self.n_tokens = n_layers, n_channels, n_tokens
        self.chunk_tokens, self.cdf_chunks = chunk_tokens, cdf_chunks

    @property
    def ref(self):
        return ctypes.byref(self.c)

    def _q(self, name):
        v = getattr(_load(), name)(self.ref)
        if v < 0:
            raise KvcError(name, int(v))
        return int(v)

    @property
    def alphabet(self): return self._q("kvc_alphabet")
    @property
    def n_chunks(self): return self._q("kvc_n_chunks")
    @property
    def n_slabs(self): return self._q("kvc_n_slabs")
    @property
    def n_streams(self): return self._q("kvc_n_streams")
    @property
    def decode_lanes(self): return self._q("kvc_decode_lanes")
    @property
    def cdf_bytes(self): return self._q("kvc_cdf_bytes")
    @property
    def scratch_bytes(self): return self._q("kvc_scratch_bytes")
    @property
    def max_payload_bytes(self): return self._q("kvc_max_payload_bytes")
    @property
    def container_payload_offset(self): return self._q("kvc_container_payload_offset")

    def container_bytes(self, payload_bytes: int) -> int:
        v = _load().kvc_container_bytes(self.ref, payload_bytes)
        if v < 0:
            raise KvcError("kvc_container_bytes", int(v))
        return int(v)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("kvc: device tensors only (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError("kvc: tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int):
    if rc != KVC_OK:
        raise KvcError(fn, rc)


# --------------------------------------------------------------- C ABI, 1:1

def kvc_version() -> int:
    return int(_load().kvc_version())


def kvc_quantize(desc: Desc, kv, sym, max1, cdf=None, dev_status=None, stream=None):
    _check("kvc_quantize", _load().kvc_quantize(desc.ref, _ptr(kv), _ptr(sym), _ptr(max1), _ptr(cdf),
                                                _ptr(dev_status), _stream(stream)))


def kvc_quantize_levels(descs, kv, syms, max1, cdfs, dev_status=None, stream=None):
    """descs: Desc per level; syms, cdfs: device tensors per level."""
    n = len(descs)
    arr = (KvcDesc * n)(*[d.c for d in descs])  # the Desc objects keep their bins alive
    ps = (ctypes.c_void_p * n)(*[_ptr(t) for t in syms])
    pc = (ctypes.c_void_p * n)(*[_ptr(t) for t in cdfs])
    _check("kvc_quantize_levels", _load().kvc_quantize_levels(arr, n, _ptr(kv), ps, _ptr(max1), pc,
                                                              _ptr(dev_status), _stream(stream)))


def kvc_cdf(desc: Desc, sym, cdf, dev_status=None, stream=None):
    _check("kvc_cdf", _load().kvc_cdf(desc.ref, _ptr(sym), _ptr(cdf), _ptr(dev_status), _stream(stream)))


def kvc_encode(desc: Desc, sym, cdf, scratch, stream_len, slab_off, payload, dev_status=None,
               stream=None, scratch_bytes=None, payload_cap=None):
    sb = scratch.numel() * scratch.element_size() if scratch_bytes is None else scratch_bytes
    pc = payload.numel() * payload.element_size() if payload_cap is None else payload_cap
    _check("kvc_encode", _load().kvc_encode(desc.ref, _ptr(sym), _ptr(cdf), _ptr(scratch), sb,
                                            _ptr(stream_len), _ptr(slab_off), _ptr(payload), pc,
                                            _ptr(dev_status), _stream(stream)))


def kvc_encode_noalloc(desc: Desc, sym, cdf, stream_len, slab_off, payload, dev_status=None, stream=None,
                       payload_cap=None):
    pc = payload.numel() * payload.element_size() if payload_cap is None else payload_cap
    _check("kvc_encode_noalloc", _load().kvc_encode_noalloc(desc.ref, _ptr(sym), _ptr(cdf), _ptr(stream_len),
                                                            _ptr(slab_off), _ptr(payload), pc,
                                                            _ptr(dev_status), _stream(stream)))


def kvc_decode(desc: Desc, payload, slab_off, stream_len, cdf, max1=None, sym_out=None, out=None,
               out_dtype=KVC_F16, dev_status=None, stream=None, payload_bytes=None):
    pb = payload.numel() * payload.element_size() if payload_bytes is None else payload_bytes
    _check("kvc_decode", _load().kvc_decode(desc.ref, _ptr(payload), pb, _ptr(slab_off),
                                            _ptr(stream_len), _ptr(cdf), _ptr(max1), _ptr(sym_out),
                                            _ptr(out), out_dtype, _ptr(dev_status), _stream(stream)))


def kvc_dequantize(desc: Desc, sym, max1, out, out_dtype=KVC_F16, stream=None):
    _check("kvc_dequantize", _load().kvc_dequantize(desc.ref, _ptr(sym), _ptr(max1), _ptr(out),
                                                    out_dtype, _stream(stream)))


def kvc_serialize(desc: Desc, cdf, max1, stream_len, slab_off, payload, out, dev_status=None,
                  stream=None, out_cap=None):
    oc = out.numel() * out.element_size() if out_cap is None else out_cap
    _check("kvc_serialize", _load().kvc_serialize(desc.ref, _ptr(cdf), _ptr(max1), _ptr(stream_len),
                                                  _ptr(slab_off), _ptr(payload), _ptr(out), oc,
                                                  _ptr(dev_status), _stream(stream)))


def kvc_serialize_chunk(desc: Desc, chunk: int, cdf, max1, stream_len, slab_off, payload, out,
                        dev_status=None, stream=None, out_cap=None):
    oc = out.numel() * out.element_size() if out_cap is None else out_cap
    _check("kvc_serialize_chunk", _load().kvc_serialize_chunk(desc.ref, chunk, _ptr(cdf), _ptr(max1),
                                                              _ptr(stream_len), _ptr(slab_off),
                                                              _ptr(payload), _ptr(out), oc,
                                                              _ptr(dev_status), _stream(stream)))


def kvc_stream_work_bytes(descs, chunks_per_unit: int = 0) -> int:
    n = len(descs)
    arr = (KvcDesc * n)(*[d.c for d in descs])
    v = int(_load().kvc_stream_work_bytes(arr, n, chunks_per_unit))
    if v < 0:
        raise KvcError("kvc_stream_work_bytes", v)
    return v


def _host_ptr(t) -> int:
    if t.is_cuda or not t.is_pinned() or not t.is_contiguous():
        raise ValueError("kvc: page-locked contiguous host tensors only (torch pin_memory)")
    return t.data_ptr()


def kvc_stream_encode(descs, chunk_level, syms, cdfs, max1, work, host_out, chunk_bytes, dev_status=None,
                      compute_stream=None, copy_stream=None, chunks_per_unit: int = 0, on_chunk=None,
                      work_bytes=None, host_cap=None):
    """descs: Desc per level; chunk_level: host int32 [NC]; syms, cdfs: device
    tensors per level; work: device buffer; host_out (uint8) and chunk_bytes
    (int64 [NC]): pinned host tensors; on_chunk(chunk, level, memoryview) or
    None.  Returns once every container is in host_out."""
    import torch
    n = len(descs)
    arr = (KvcDesc * n)(*[d.c for d in descs])
    ps = (ctypes.c_void_p * n)(*[_ptr(t) for t in syms])
    pc = (ctypes.c_void_p * n)(*[_ptr(t) for t in cdfs])
    lv = np.ascontiguousarray(np.asarray(chunk_level, dtype=np.int32))
    wb = work.numel() * work.element_size() if work_bytes is None else work_bytes
    hc = host_out.numel() * host_out.element_size() if host_cap is None else host_cap
    if chunk_bytes.dtype != torch.int64:
        raise ValueError("kvc: chunk_bytes must be int64")
    if on_chunk is None:
        cb = ctypes.cast(None, CHUNK_FN)
    else:
        def _cb(_user, chunk, level, ptr, nbytes):
            on_chunk(int(chunk), int(level), (ctypes.c_uint8 * nbytes).from_address(ptr))
        cb = CHUNK_FN(_cb)
    cs = _stream(compute_stream)
    xs = cs if copy_stream is None else _stream(copy_stream)
    _check("kvc_stream_encode", _load().kvc_stream_encode(
        arr, n, lv.ctypes.data, ps, pc, _ptr(max1), chunks_per_unit, _ptr(work), wb, _host_ptr(host_out), hc,
        _host_ptr(chunk_bytes), _ptr(dev_status), cs, xs, cb, None))


def kvc_deserialize(desc: Desc, inp, cdf, max1, stream_len, slab_off, dev_status=None, stream=None,
                    in_bytes=None):
    nb = inp.numel() * inp.element_size() if in_bytes is None else in_bytes
    _check("kvc_deserialize", _load().kvc_deserialize(desc.ref, _ptr(inp), nb, _ptr(cdf), _ptr(max1),
                                                      _ptr(stream_len), _ptr(slab_off),
                                                      _ptr(dev_status), _stream(stream)))


def kvc_int8_quantize(desc: Desc, group: int, kv, q, scale, zero_point, dev_status=None,
                      stream=None):
    _check("kvc_int8_quantize", _load().kvc_int8_quantize(desc.ref, group, _ptr(kv), _ptr(q),
                                                          _ptr(scale), _ptr(zero_point),
                                                          _ptr(dev_status), _stream(stream)))


def kvc_int8_dequantize(desc: Desc, group: int, q, scale, zero_point, out, out_dtype=KVC_F16, stream=None):
    _check("kvc_int8_dequantize", _load().kvc_int8_dequantize(desc.ref, group, _ptr(q), _ptr(scale),
                                                              _ptr(zero_point), _ptr(out), out_dtype,
                                                              _stream(stream)))


def kvc_delta_forward(desc: Desc, anchor_tokens: int, kv, delta, dev_status=None, stream=None):
    _check("kvc_delta_forward", _load().kvc_delta_forward(desc.ref, anchor_tokens, _ptr(kv), _ptr(delta),
                                                          _ptr(dev_status), _stream(stream)))


def kvc_delta_inverse(desc: Desc, anchor_tokens: int, y, stream=None):
    _check("kvc_delta_inverse", _load().kvc_delta_inverse(desc.ref, anchor_tokens, _ptr(y), _stream(stream)))


# --------------------------------------------------------------- convenience

@dataclass
class Buffers:
    """Preallocated device buffers for one problem shape."""
    desc: Desc
    sym: "object"
    max1: "object"
    cdf: "object"
    scratch: "object"
    stream_len: "object"
    slab_off: "object"
    payload: "object"
    dev_status: "object"
    out: "object"
    dec_sym: "object"


def alloc(desc: Desc, device="cuda", out_dtype=KVC_F16, with_dec_sym=False) -> Buffers:
    import torch
    L, C, T = desc.n_layers, desc.n_channels, desc.n_tokens
    u8, u16, i64 = torch.uint8, torch.int16, torch.int64

    def z(n, dt):
        return torch.empty(max(n, 1), dtype=dt, device=device)

    odt = torch.float16 if out_dtype == KVC_F16 else torch.float32
    n_el = L * 2 * T * C
    return Buffers(
        desc=desc,
        sym=z(n_el, u8), max1=z(L * 2 * T, u16),
        cdf=z(desc.cdf_bytes // 2, u16),
        scratch=z((desc.scratch_bytes + 15) // 16 * 16, u8),
        stream_len=z(desc.n_streams, u16),
        slab_off=z(desc.n_slabs + 1, i64),
        payload=z((desc.max_payload_bytes + 15) // 16 * 16, u8),
        dev_status=torch.zeros(1, dtype=torch.int32, device=device),
        out=z(n_el, odt),
        dec_sym=z(n_el, u8) if with_dec_sym else None,
    )


def encode(buf: Buffers, kv, fused_cdf: bool = True, stream=None):
    """quantize (+ CDF) then range-code and pack, all on `stream`."""
    d = buf.desc
    kvc_quantize(d, kv, buf.sym, buf.max1, buf.cdf if fused_cdf else None, buf.dev_status, stream)
    if not fused_cdf:
        kvc_cdf(d, buf.sym, buf.cdf, buf.dev_status, stream)
    kvc_encode(d, buf.sym, buf.cdf, buf.scratch, buf.stream_len, buf.slab_off, buf.payload,
               buf.dev_status, stream)


def decode(buf: Buffers, out_dtype=KVC_F16, stream=None, payload=None, payload_bytes=None):
    """decode + fused dequantize into buf.out (and buf.dec_sym if allocated)."""
    d = buf.desc
    kvc_decode(d, buf.payload if payload is None else payload, buf.slab_off, buf.stream_len, buf.cdf,
               buf.max1, buf.dec_sym, buf.out, out_dtype, buf.dev_status, stream,
               payload_bytes=payload_bytes)


# --------------------------------------------------- the resident 4-bit cache

class Kv4Cache:
    """One layer's paged 4-bit K/V pool: a kvc_kv4_desc, its two device buffers
    and a status word.  Layouts as in kvc.h: codes uint8
    [n_pages][2][H][P * D/2], params float16 [n_pages][2][H][D/G][P][2] (s, lo).
    Another tensor may be assigned to any of the three; it is checked as the first was."""

    def __init__(self, n_kv_heads: int, head_dim: int, n_pages: int, page_tokens: int = 64, group: int = 64,
                 codes=None, params=None, dev_status=None, device="cuda"):
        import torch
        self.c = KvcKv4Desc(n_kv_heads, head_dim, group, page_tokens, n_pages)
        self.ref = ctypes.byref(self.c)
        self.n_kv_heads, self.head_dim, self.group = n_kv_heads, head_dim, group
        self.page_tokens, self.n_pages = page_tokens, n_pages
        self.int32, self.int64, self.float32 = torch.int32, torch.int64, torch.float32
        self._want = {}  # type and bytes of a buffer
        for name, dt in (("codes", torch.uint8), ("params", torch.float16)):
            v = int(getattr(_load(), f"kvc_kv4_{name}_bytes")(self.ref))
            if v < 0:
                raise KvcError(f"kvc_kv4_{name}_bytes", v)
            self._want[name] = dt, v
        given = [t for t in (codes, params, dev_status) if t is not None]
        device = given[0].device if given else device
        if codes is None:
            codes = torch.empty((n_pages, 2, n_kv_heads, page_tokens * head_dim // 2), dtype=torch.uint8, device=device)
        if params is None:
            params = torch.empty((n_pages, 2, n_kv_heads, head_dim // group, page_tokens, 2), dtype=torch.float16,
                                 device=device)
        self.device_index = codes.get_device()
        self.codes, self.params = codes, params
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=codes.device) if dev_status is None else dev_status

    # The calls take the address of each, kept beside it.

    @property
    def codes(self):
        return self._codes

    @codes.setter
    def codes(self, t):
        self._codes, self.codes_ptr = t, self._checked("codes", t)

    @property
    def params(self):
        return self._params

    @params.setter
    def params(self, t):
        self._params, self.params_ptr = t, self._checked("params", t)

    @property
    def dev_status(self):
        return self._status

    @dev_status.setter
    def dev_status(self, t):
        if t.dtype != self.int32 or t.numel() < 1:
            raise ValueError("kvc: dev_status must be torch.int32")
        if t.get_device() != self.device_index:
            raise _wrong_device("dev_status", t)
        self._status, self.status_ptr = t, _ptr(t)

    def _checked(self, name, t):
        dt, nb = self._want[name]
        if t.dtype != dt or t.numel() * t.element_size() != nb:
            raise ValueError(f"kvc: {name} must be {dt} of {nb} bytes")
        if t.get_device() != self.device_index:
            raise _wrong_device(name, t)
        return _ptr(t)


_KV4_DTYPES = {}  # torch.dtype -> KVC_* (filled on first use: torch is imported late)
_ATTN = struct.Struct("@PPPqqqqPqPPqiiiiiiiffPq")  # kvc_kv4_attn, field by field as KvcKv4Attn
_RAW_STREAM = _CURRENT_DEVICE = None


def _kv4_dtype(dt):
    v = _KV4_DTYPES.get(dt)
    if v is None:
        import torch
        _KV4_DTYPES.update({torch.float16: KVC_F16, torch.float32: KVC_F32, torch.bfloat16: KVC_BF16})
        v = _KV4_DTYPES.get(dt)
        if v is None:
            raise ValueError(f"kvc: float16, bfloat16 or float32, not {dt}")
    return v


def _wrong_device(name, t):
    return ValueError(f"kvc: {name} must be on the cache's device" if t.is_cuda else
                      "kvc: device tensors only (there is no CPU path)")


def _kv4_call(fn, cache, stream, *args):
    """Launches on the caller's stream, or the current one of the cache's device (without building a
    torch.cuda.Stream: these calls are a few microseconds long), with that device current."""
    global _RAW_STREAM, _CURRENT_DEVICE
    if _RAW_STREAM is None:
        import torch
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)
        _CURRENT_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    dev = cache.device_index
    stream = _RAW_STREAM(dev) if stream is None else _stream(stream)
    if _CURRENT_DEVICE() == dev:
        return fn(cache.ref, *args, stream)
    import torch
    with torch.cuda.device(dev):
        return fn(cache.ref, *args, stream)


def _kv4_empty(stream, like, shape, dtype):
    """A tensor for the kernels of a call on `stream`, of that stream's memory: the current stream's could be in use
    there still, or be given away before the kernels are done with it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, like.device) if stream else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _rows(name: str, t, shape, dev: int, written=False):
    """Pointer and strides of a device tensor [n][heads][D] whose channels are contiguous; one that is written
    may not have rows in each other's place (an expanded tensor)."""
    if t.shape != shape:
        raise ValueError(f"kvc: {name} must be {list(shape)}, not {list(t.shape)}")
    if t.get_device() != dev:
        raise _wrong_device(name, t)
    ts, hs, cs = t.stride()
    if cs != 1:
        raise ValueError(f"kvc: the channels of {name} must be contiguous")
    if written and (-shape[2] < ts < shape[2] and shape[0] > 1 or -shape[2] < hs < shape[2] and shape[1] > 1):
        raise ValueError(f"kvc: the rows of {name} overlap")
    return t.data_ptr(), ts, hs


def _ints(name: str, t, dt, shape, dev: int):
    if t.dtype != dt or t.shape != shape:
        raise ValueError(f"kvc: {name} must be {dt} of shape {list(shape)}, not {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise _wrong_device(name, t)
    if not t.is_contiguous():
        raise ValueError("kvc: tensors must be contiguous")
    return t.data_ptr()


def kv4_append(cache: Kv4Cache, k, v, slots, stream=None):
    """Quantise k, v [T][H][D] (float16, bfloat16 or float32) into the slots
    int64 [T] (page * page_tokens + token in page; negative: skipped)."""
    n, dev = k.shape[0], cache.device_index
    if v.dtype != k.dtype:
        raise ValueError("kvc: k and v must have one dtype")
    shape = (n, cache.n_kv_heads, cache.head_dim)
    kp, kts, khs = _rows("k", k, shape, dev)
    vp, vts, vhs = _rows("v", v, shape, dev)
    rc = _kv4_call(_load().kvc_kv4_append, cache, stream, kp, vp, n, kts, khs, vts, vhs, _kv4_dtype(k.dtype),
                   _ints("slots", slots, cache.int64, (n,), dev), cache.codes_ptr, cache.params_ptr, cache.status_ptr)
    if rc:
        raise KvcError("kvc_kv4_append", rc)


def kv4_read(cache: Kv4Cache, slots, dtype=None, k=None, v=None, stream=None):
    """The values at slots int64 [T], as (k, v) [T][H][D] of `dtype` (float16
    unless given) or written into k and v (one dtype, channels contiguous).
    What is allocated here belongs to `stream` (the current one if not given)."""
    if slots.dim() != 1:
        raise ValueError("kvc: slots must be int64 [T]")
    n, dev = slots.shape[0], cache.device_index
    if dtype is None:
        dtype = cache.params.dtype if k is None and v is None else (v if k is None else k).dtype
    shape = (n, cache.n_kv_heads, cache.head_dim)
    if k is None:
        k = slots.new_empty(shape, dtype=dtype) if stream is None else _kv4_empty(stream, slots, shape, dtype)
    if v is None:
        v = slots.new_empty(shape, dtype=dtype) if stream is None else _kv4_empty(stream, slots, shape, dtype)
    if k.dtype != dtype or v.dtype != dtype:
        raise ValueError("kvc: k and v must have one dtype")
    kp, kts, khs = _rows("k", k, shape, dev, True)
    vp, vts, vhs = _rows("v", v, shape, dev, True)
    rc = _kv4_call(_load().kvc_kv4_read, cache, stream, cache.codes_ptr, cache.params_ptr,
                   _ints("slots", slots, cache.int64, (n,), dev), n, kp, vp, kts, khs, vts, vhs, _kv4_dtype(dtype),
                   cache.status_ptr)
    if rc:
        raise KvcError("kvc_kv4_read", rc)
    return k, v


def kv4_work_bytes(cache: Kv4Cache, n_q: int, n_q_heads: int, n_seqs: int, max_pages: int, max_q: int) -> int:
    """Workspace of a kv4_attention call: n_q query tokens in all, at most
    max_q of one sequence, page tables of max_pages entries."""
    v = int(_load().kvc_kv4_work_bytes(cache.ref, n_q, n_seqs, n_q_heads, max_pages, max_q))
    if v < 0:
        raise KvcError("kvc_kv4_work_bytes", v)
    return v


def kv4_attention(cache: Kv4Cache, q, page_table, kv_len, cu_q=None, max_q: Optional[int] = None, causal: bool = True,
                  window: int = 0, softcap: float = 0.0, scale: Optional[float] = None, out=None,
                  return_lse: bool = False, lse=None, work=None, stream=None):
    """Attention of q [n_q][Hq][D] (float16 or bfloat16) over the cached keys:
    the last query of sequence b stands at its last key.  page_table int32
    [B][max_pages], kv_len int32 [B]; cu_q int32 [B + 1] bounds each
    sequence's queries (at most max_q, by which the launch is planned; n_q if
    not given; rows outside all of them are not written), without it every
    sequence has n_q / B.  `work`: uint8 of kv4_work_bytes, allocated if not
    given.  What is allocated here belongs to `stream` (the current one if not
    given).  Returns out, or (out, lse float32 [n_q][Hq])."""
    if q.dim() != 3 or page_table.dim() != 2:
        raise ValueError("kvc: q must be [n_q][Hq][D], page_table [B][max_pages]")
    n_q, n_heads, _ = q.shape
    shape = (n_q, n_heads, cache.head_dim)
    B, max_pages = page_table.shape
    i32, f32, dtype, dev = cache.int32, cache.float32, q.dtype, cache.device_index
    if page_table.dtype != i32 or (max_pages > 1 and page_table.stride(1) != 1):
        raise ValueError("kvc: page_table must be a device int32 tensor with contiguous rows")
    if page_table.get_device() != dev:
        raise _wrong_device("page_table", page_table)
    if cu_q is None:
        if B == 0 or n_q % B:
            raise ValueError("kvc: without cu_q every sequence has the same number of queries")
        if max_q is not None and max_q != n_q // B:
            raise ValueError("kvc: without cu_q max_q is n_q / B")
        max_q = n_q // B
    elif max_q is None:
        max_q = n_q
    if out is None:
        out = q.new_empty(shape) if stream is None else _kv4_empty(stream, q, shape, dtype)
    elif out.dtype != dtype:
        raise ValueError("kvc: out must have q's dtype")
    if lse is not None:
        return_lse = True
    elif return_lse:
        lse = q.new_empty(shape[:2], dtype=f32) if stream is None else _kv4_empty(stream, q, shape[:2], f32)
    if work is None:
        nb = kv4_work_bytes(cache, n_q, n_heads, B, max_pages, max_q)
        work = _kv4_empty(stream, q, (nb,), cache.codes.dtype) if nb else None
    elif work.get_device() != dev:
        raise _wrong_device("work", work)
    qp, qts, qhs = _rows("q", q, shape, dev)
    op, ots, ohs = _rows("out", out, shape, dev, True)
    args = _ATTN.pack(
        qp, op, 0 if lse is None else _ints("lse", lse, f32, shape[:2], dev), qts, qhs, ots, ohs,
        page_table.data_ptr(), page_table.stride(0),
        _ints("kv_len", kv_len, i32, (B,), dev), 0 if cu_q is None else _ints("cu_q", cu_q, i32, (B + 1,), dev),
        n_q, B, n_heads, max_pages, max_q, _kv4_dtype(dtype), bool(causal), window, softcap,
        cache.head_dim ** -0.5 if scale is None else scale, 0 if work is None else _ptr(work),
        0 if work is None else work.numel() * work.element_size())
    rc = _kv4_call(_load().kvc_kv4_attention, cache, stream, args, cache.codes_ptr, cache.params_ptr, cache.status_ptr)
    if rc:
        raise KvcError("kvc_kv4_attention", rc)
    return (out, lse) if return_lse else out
