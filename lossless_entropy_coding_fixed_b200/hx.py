"""Python binding of the hx C ABI (include/hx.h): argument marshalling only.

Every step of the coder runs in libhx.so: the codebook builder on the host, the histogram,
encode and decode kernels on the GPU. PyTorch supplies device memory and the current CUDA
stream; tensors are passed as raw pointers. There is no fallback: if the library is missing or
cannot load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from dataclasses import dataclass

import numpy as np

from . import build as _build

HX_OK, HX_ERR_ARG, HX_ERR_CUDA = 0, 1, 2
HX_ERR_UNCODABLE, HX_ERR_CORRUPT, HX_ERR_CODEBOOK, HX_ERR_TIMEOUT, HX_ERR_CAPACITY = 4, 8, 16, 32, 64
KIND_HUFFMAN, KIND_QLC, KIND_SHANNONIC, KIND_EXPGOLOMB = 0, 1, 2, 3
CHUNK, SUBSTREAMS, LMAX_MAX, QLC_LMAX = 4096, 8, 12, 11
CB_SEEN_ONLY = 1
TABLES_BYTES = 10240
F32, F16, BF16 = 0, 1, 2
ROWS_E4M3, ROWS_INT8 = 0, 1

HEADER = os.path.join(_build.INCLUDE, "hx.h")


class HxError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: status {code} ({status_string(code)})")
        self.code = code


class _Codebook(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_uint8), ("lmax", ctypes.c_uint8),
                ("len", ctypes.c_uint8 * 256), ("code", ctypes.c_uint16 * 256),
                ("qlc_bits", ctypes.c_uint8 * 8), ("qlc_start", ctypes.c_uint16 * 9),
                ("rank2sym", ctypes.c_uint8 * 256), ("hash", ctypes.c_uint64),
                ("sh_nr", ctypes.c_uint8), ("sh_lo", ctypes.c_uint16 * 17),
                ("sh_f", ctypes.c_uint8 * 16)]


_lib = None


def declared_functions() -> list[str]:
    """Names of the functions include/hx.h declares."""
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.findall(r"^\s*(?:int|uint64_t|double|const char\*)\s+(hx_\w+)\s*\(", text,
                      flags=re.M)


def lib():
    """Load libhx.so (building it first when the sources are newer). Raises if it cannot."""
    global _lib
    if _lib is None:
        if not _build.up_to_date():
            _build.build()
        L = ctypes.CDLL(_build.LIB)
        P, u64, i32, u32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_uint32
        CB = ctypes.POINTER(_Codebook)
        sig = {
            "hx_build_codebook": (i32, [P, i32, u32, CB]),
            "hx_qlc_build": (i32, [P, i32, u32, CB]),
            "hx_codebook_tables": (i32, [CB, P]),
            "hx_codebook_upload": (i32, [CB, P, P]),
            "hx_histogram": (i32, [P, u64, P, P]),
            "hx_payload_offset": (u64, [u64]),
            "hx_sync_offset": (u64, [u64]),
            "hx_encode_bound": (u64, [u64]),
            "hx_scratch_bytes": (u64, [u64]),
            "hx_encode": (i32, [P, P, u64, P, u64, P, P, P, P]),
            "hx_decode": (i32, [P, P, u64, P, u64, P, P]),
            "hx_qlc_encode": (i32, [P, P, u64, P, u64, P, P, P, P]),
            "hx_qlc_decode": (i32, [P, P, u64, P, u64, P, P]),
            "hx_encode_noalloc": (i32, [P, P, u64, P, u64, P, P, P]),
            "hx_encode_bounded": (i32, [u32, P, P, u64, P, u64, P, P, P, u64, u64, u32, P]),
            "hx_shannonic_build": (i32, [P, i32, u32, CB]),
            "hx_expgolomb_build": (i32, [i32, i32, CB]),
            "hx_expgolomb_encode": (i32, [P, P, u64, P, u64, P, P, P, P]),
            "hx_expgolomb_decode": (i32, [P, P, u64, P, u64, P, P]),
            "hx_shannonic_encode_bound": (u64, [u64]),
            "hx_shannonic_encode": (i32, [P, P, u64, P, u64, P, P, P, P]),
            "hx_shannonic_decode": (i32, [P, P, u64, P, u64, P, P]),
            "hx_decode_set": (i32, [u32, P, u32, P, u64, P, u64, P, P]),
            "hx_planner_create": (i32, [ctypes.POINTER(_SessionConfig), P, P]),
            "hx_planner_codebook": (i32, [P, u64, CB]),
            "hx_planner_observe": (i32, [P, u64, P, P, P]),
            "hx_planner_destroy": (None, [P]),
            "hx_session_create": (i32, [ctypes.POINTER(_SessionConfig), P, P, u32, P]),
            "hx_session_encode": (i32, [P, P, u64, P, u64, P, P, P, P]),
            "hx_session_decode": (i32, [P, P, u64, P, u64, P, P]),
            "hx_session_drain": (i32, [P]),
            "hx_session_batch_info": (i32, [P, u64, ctypes.POINTER(_BatchInfo)]),
            "hx_session_destroy": (None, [P]),
            "hx_quantize_rows": (i32, [u32, u32, P, u64, u64, u64, P, P, P]),
            "hx_dequantize_rows": (i32, [u32, u32, P, P, u64, u64, P, u64, P]),
            "hx_gated_forward": (i32, [u32, u32, P, u64, u64, u64, P, P, P, P]),
            "hx_gated_backward": (i32, [u32, u32, P, u64, P, P, u64, u64, P, P, P]),
            "hx_head_norm_rope_forward": (i32, [P, P, u64, u64, P, u64, u64,
                                                P, P, P, P]),
            "hx_head_norm_rope_workspace": (u64, [u32]),
            "hx_head_norm_rope_backward": (i32, [P, P, u64, u64, P, P, P, u64,
                                                 u64, P, P, P, u64, P, P]),
            "hx_weight_grad_workspace": (u64, [P, u64, P, u64, u64, u64]),
            "hx_weight_grad": (i32, [u32, u32, P, u64, P, P, u64, u64, u64, u32, P, u64, i32, P, u64, P, P]),
            "hx_weight_grad_bounded": (i32, [u32, u32, P, u64, P, P, u64, u64, u64, u32, P, u64, i32, P, u64, P, u64, u64, P]),
            "hx_entropy": (ctypes.c_double, [P]),
            "hx_mean_length": (ctypes.c_double, [P, CB]),
            "hx_version": (i32, []),
            "hx_status_string": (ctypes.c_char_p, [i32]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().hx_status_string(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc:
        raise HxError(rc, what)


class _HeadNormRope(ctypes.Structure):
    _fields_ = [("format", ctypes.c_uint32), ("dtype", ctypes.c_uint32),
                ("weight_dtype", ctypes.c_uint32), ("position_bits", ctypes.c_uint32),
                ("tokens", ctypes.c_uint64), ("q_heads", ctypes.c_uint32),
                ("k_heads", ctypes.c_uint32), ("dim", ctypes.c_uint32), ("rot_dim", ctypes.c_uint32),
                ("interleaved", ctypes.c_uint32), ("eps", ctypes.c_float), ("places", ctypes.c_uint64),
                ("d_wq", ctypes.c_void_p), ("d_wk", ctypes.c_void_p), ("d_cos", ctypes.c_void_p),
                ("d_sin", ctypes.c_void_p), ("d_positions", ctypes.c_void_p)]


class _SessionConfig(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_uint32), ("lmax", ctypes.c_uint32),
                ("max_distinct", ctypes.c_uint32), ("flags", ctypes.c_uint32),
                ("history", ctypes.c_uint32), ("lag", ctypes.c_uint32), ("drift", ctypes.c_double)]


class _BatchInfo(ctypes.Structure):
    _fields_ = [("hash", ctypes.c_uint64), ("slot", ctypes.c_uint32), ("observed", ctypes.c_int32),
                ("refreshed", ctypes.c_int32), ("pad", ctypes.c_uint32),
                ("symbols", ctypes.c_uint64), ("drift", ctypes.c_double)]


# ------------------------------------------------------------------------------ codebooks (host)
@dataclass
class Codebook:
    """A host codebook (hx_codebook)."""
    raw: _Codebook

    @property
    def kind(self) -> int:
        return self.raw.kind

    @property
    def lmax(self) -> int:
        return self.raw.lmax

    @property
    def len(self) -> np.ndarray:
        return np.frombuffer(bytes(self.raw.len), np.uint8).copy()

    @property
    def code(self) -> np.ndarray:
        return np.frombuffer(bytes(self.raw.code), np.uint16).copy()

    @property
    def qlc_bits(self) -> np.ndarray:
        return np.frombuffer(bytes(self.raw.qlc_bits), np.uint8).copy()

    @property
    def qlc_start(self) -> np.ndarray:
        return np.frombuffer(bytes(self.raw.qlc_start), np.uint16).copy()

    @property
    def rank2sym(self) -> np.ndarray:
        return np.frombuffer(bytes(self.raw.rank2sym), np.uint8).copy()

    @property
    def hash(self) -> int:
        return int(self.raw.hash)

    @property
    def sh_lo(self) -> np.ndarray:
        return np.frombuffer(bytes(self.raw.sh_lo), np.uint16)[: self.raw.sh_nr + 1].copy()

    @property
    def sh_f(self) -> np.ndarray:
        return np.frombuffer(bytes(self.raw.sh_f), np.uint8)[: self.raw.sh_nr].copy()

    def tables(self) -> bytes:
        buf = (ctypes.c_uint8 * TABLES_BYTES)()
        _check(lib().hx_codebook_tables(ctypes.byref(self.raw), buf), "hx_codebook_tables")
        return bytes(buf)

    def upload(self, device=None):
        """The table block as a device uint8 tensor (HX_TABLES_BYTES), copied on the current stream."""
        import torch
        t = torch.empty(TABLES_BYTES, dtype=torch.uint8, device=device or "cuda")
        _check(lib().hx_codebook_upload(ctypes.byref(self.raw), t.data_ptr(), _stream(t)),
               "hx_codebook_upload")
        return t


def _counts(counts) -> np.ndarray:
    c = np.ascontiguousarray(np.asarray(counts, dtype=np.uint64).reshape(-1))
    if c.size != 256:
        raise ValueError("counts must have 256 entries")
    return c


def build_codebook(counts, lmax: int = 12, seen_only: bool = False) -> Codebook:
    c = _counts(counts)
    raw = _Codebook()
    _check(lib().hx_build_codebook(c.ctypes.data, int(lmax), CB_SEEN_ONLY if seen_only else 0,
                                   ctypes.byref(raw)), "hx_build_codebook")
    return Codebook(raw)


def qlc_build(counts, max_distinct: int = 4) -> Codebook:
    c = _counts(counts)
    raw = _Codebook()
    _check(lib().hx_qlc_build(c.ctypes.data, int(max_distinct), 0, ctypes.byref(raw)),
           "hx_qlc_build")
    return Codebook(raw)


def shannonic_build(counts, K: int = 16) -> Codebook:
    """hx_shannonic_build: range partition (at most K ranges) and 128-state tANS frequencies."""
    c = _counts(counts)
    raw = _Codebook()
    _check(lib().hx_shannonic_build(c.ctypes.data, int(K), 0, ctypes.byref(raw)),
           "hx_shannonic_build")
    return Codebook(raw)


def expgolomb_build(order: int = 5, map: int = 0) -> Codebook:
    """hx_expgolomb_build: Exp-Golomb of order 5..8 over a sign/magnitude (map 0) or zigzag
    (map 1) index of the byte."""
    raw = _Codebook()
    _check(lib().hx_expgolomb_build(int(order), int(map), ctypes.byref(raw)), "hx_expgolomb_build")
    return Codebook(raw)


def entropy(counts) -> float:
    """Shannon entropy of a 256-bin histogram, bits per symbol."""
    c = _counts(counts)
    return float(lib().hx_entropy(c.ctypes.data))


def mean_length(counts, cb: Codebook) -> float:
    """Mean code length (bits per symbol) of `cb` on data with this histogram."""
    c = _counts(counts)
    return float(lib().hx_mean_length(c.ctypes.data, ctypes.byref(cb.raw)))


# ------------------------------------------------------------------------------ layout helpers
def payload_offset(n: int) -> int:
    return int(lib().hx_payload_offset(n))


def sync_offset(n: int) -> int:
    return int(lib().hx_sync_offset(n))


def encode_bound(n: int, kind: int = KIND_HUFFMAN) -> int:
    if kind == KIND_SHANNONIC:
        return int(lib().hx_shannonic_encode_bound(n))
    return int(lib().hx_encode_bound(n))


def scratch_bytes(n: int) -> int:
    return int(lib().hx_scratch_bytes(n))


def stream_bytes(n: int, total_words: int) -> int:
    return payload_offset(n) + 4 * (int(total_words) + 2)


# ------------------------------------------------------------------------------ device calls
def _stream(t) -> int:
    import torch
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev_u8(x, what):
    import torch
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.uint8 and x.is_contiguous()):
        raise TypeError(f"{what} must be a contiguous CUDA uint8 tensor")
    return x


def new_status(device=None):
    import torch
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def histogram(x, counts=None):
    """counts (int32[256] on the device) += histogram of x; returns counts."""
    import torch
    x = _dev_u8(x, "x")
    if counts is None:
        counts = torch.zeros(256, dtype=torch.int32, device=x.device)
    _check(lib().hx_histogram(x.data_ptr(), x.numel(), counts.data_ptr(), _stream(x)), "hx_histogram")
    return counts


def encode(tables, x, out=None, scratch=None, hist=None, status=None, kind: int = KIND_HUFFMAN):
    """Encode device bytes x with the device table block `tables`.

    Returns (out, status): out holds the stream (its first stream_size(out, n) bytes are
    meaningful), status is the device status word (0 when every check passed)."""
    import torch
    x = _dev_u8(x, "x")
    n = x.numel()
    if out is None:
        out = torch.empty(encode_bound(n, kind), dtype=torch.uint8, device=x.device)
    if scratch is None:
        scratch = torch.empty(scratch_bytes(n), dtype=torch.uint8, device=x.device)
    if status is None:
        status = new_status(x.device)
    fn = {KIND_HUFFMAN: lib().hx_encode, KIND_QLC: lib().hx_qlc_encode,
          KIND_SHANNONIC: lib().hx_shannonic_encode, KIND_EXPGOLOMB: lib().hx_expgolomb_encode}[kind]
    _check(fn(tables.data_ptr(), x.data_ptr(), n, out.data_ptr(), out.numel(), scratch.data_ptr(),
              hist.data_ptr() if hist is not None else None, status.data_ptr(), _stream(x)),
           "hx_encode")
    return out, status


def encode_bounded(tables, x, out, scratch, wait_ns: int, withhold: int = (1 << 64) - 1,
                   hist=None, status=None, kind: int = KIND_HUFFMAN, flush_rounds: int = 0):
    """hx_encode_bounded: encode() with the chunks' wait limit in nanoseconds and, for failure
    tests, one chunk (`withhold`) that never publishes its word count; `flush_rounds` is the
    chunks a warp codes between its flushes of the fused histogram (0: the default). Returns
    (out, status)."""
    x = _dev_u8(x, "x")
    out = _dev_u8(out, "out")
    if status is None:
        status = new_status(x.device)
    _check(lib().hx_encode_bounded(kind, tables.data_ptr(), x.data_ptr(), x.numel(),
                                   out.data_ptr(), out.numel(), scratch.data_ptr(),
                                   hist.data_ptr() if hist is not None else None,
                                   status.data_ptr(), int(wait_ns), int(withhold),
                                   int(flush_rounds), _stream(x)),
           "hx_encode_bounded")
    return out, status


NOALLOC_MAX_BYTES = 128 << 20


def encode_noalloc(tables, x, out, hist=None, status=None):
    """hx_encode_noalloc: Huffman encode whose scratch lives in the library (no allocation inside
    the call; `out` and `status` are the caller's). For callers that cannot allocate device
    memory at encode time. n <= NOALLOC_MAX_BYTES; calls overlapping on the GPU race."""
    x = _dev_u8(x, "x")
    out = _dev_u8(out, "out")
    if status is None:
        status = new_status(x.device)
    _check(lib().hx_encode_noalloc(tables.data_ptr(), x.data_ptr(), x.numel(), out.data_ptr(),
                                   out.numel(), hist.data_ptr() if hist is not None else None,
                                   status.data_ptr(), _stream(x)), "hx_encode_noalloc")
    return out, status


def decode(tables, stream, n: int, out=None, status=None, kind: int = KIND_HUFFMAN, nbytes=None):
    """Decode n bytes from the device stream. Returns (out, status)."""
    import torch
    stream = _dev_u8(stream, "stream")
    if out is None:
        out = torch.empty(max(n, 1), dtype=torch.uint8, device=stream.device)[:n]
    if status is None:
        status = new_status(stream.device)
    fn = {KIND_HUFFMAN: lib().hx_decode, KIND_QLC: lib().hx_qlc_decode,
          KIND_SHANNONIC: lib().hx_shannonic_decode, KIND_EXPGOLOMB: lib().hx_expgolomb_decode}[kind]
    _check(fn(tables.data_ptr(), stream.data_ptr(), int(nbytes or stream.numel()),
              out.data_ptr() if n else stream.data_ptr(), n, status.data_ptr(), _stream(stream)),
           "hx_decode")
    return out, status


def total_words(stream) -> int:
    """total_words from a stream header (reads 8 bytes back: synchronises with the stream)."""
    return int(np.frombuffer(stream[32:40].cpu().numpy().tobytes(), np.uint64)[0])


def stream_size(stream, n: int) -> int:
    return stream_bytes(n, total_words(stream))


MAX_TABLE_SET = 8


def decode_set(kind: int, tables, stream, n: int, out=None, status=None, nbytes=None):
    """hx_decode_set: decode with whichever of the device table blocks `tables` the stream's
    header hash names (picked on the device). Returns (out, status)."""
    import torch
    stream = _dev_u8(stream, "stream")
    if out is None:
        out = torch.empty(max(n, 1), dtype=torch.uint8, device=stream.device)[:n]
    if status is None:
        status = new_status(stream.device)
    ptrs = (ctypes.c_void_p * len(tables))(*[t.data_ptr() for t in tables])
    _check(lib().hx_decode_set(kind, ptrs, len(tables), stream.data_ptr(),
                               int(nbytes or stream.numel()),
                               out.data_ptr() if n else stream.data_ptr(), n, status.data_ptr(),
                               _stream(stream)), "hx_decode_set")
    return out, status


def _config(kind, history, lag, drift, lmax=12, max_distinct=4, seen_only=False):
    return _SessionConfig(kind=kind, lmax=lmax if kind == KIND_HUFFMAN else 0,
                          max_distinct=max_distinct if kind == KIND_QLC else 0,
                          flags=CB_SEEN_ONLY if seen_only else 0, history=history, lag=lag,
                          drift=float(drift))


class Planner:
    """hx_planner: the online loop's bookkeeping on the host (which codebook codes batch t)."""

    def __init__(self, kind=KIND_HUFFMAN, history=4, lag=2, drift=0.0, initial_counts=None,
                 **kw):
        self._cfg = _config(kind, history, lag, drift, **kw)
        init = None if initial_counts is None else _counts(initial_counts)
        h = ctypes.c_void_p()
        _check(lib().hx_planner_create(ctypes.byref(self._cfg),
                                       None if init is None else init.ctypes.data,
                                       ctypes.byref(h)), "hx_planner_create")
        self._h = h

    def codebook(self, batch: int) -> Codebook:
        raw = _Codebook()
        _check(lib().hx_planner_codebook(self._h, batch, ctypes.byref(raw)), "hx_planner_codebook")
        return Codebook(raw)

    def observe(self, batch: int, counts) -> tuple[bool, float]:
        c = _counts(counts)
        r, d = ctypes.c_int(), ctypes.c_double()
        _check(lib().hx_planner_observe(self._h, batch, c.ctypes.data, ctypes.byref(r),
                                        ctypes.byref(d)), "hx_planner_observe")
        return bool(r.value), float(d.value)

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.hx_planner_destroy(h)


class Session:
    """hx_session: encode a sequence of batches, each with the codebook of earlier batches'
    fused histograms; decode picks the table by the stream's codebook hash. The table slots,
    the histogram buffer and the status word are device tensors this object holds."""

    def __init__(self, device, kind=KIND_HUFFMAN, history=4, lag=2, drift=0.0,
                 initial_counts=None, slots=None, **kw):
        import torch
        self._cfg = _config(kind, history, lag, drift, **kw)
        self.kind = kind
        nslots = slots or min(MAX_TABLE_SET, lag + 2)
        self.slots = [torch.empty(TABLES_BYTES, dtype=torch.uint8, device=device)
                      for _ in range(nslots)]
        self.hist = torch.zeros(256, dtype=torch.int32, device=device)
        init = None if initial_counts is None else _counts(initial_counts)
        ptrs = (ctypes.c_void_p * nslots)(*[t.data_ptr() for t in self.slots])
        h = ctypes.c_void_p()
        _check(lib().hx_session_create(ctypes.byref(self._cfg),
                                       None if init is None else init.ctypes.data, ptrs, nslots,
                                       ctypes.byref(h)), "hx_session_create")
        self._h = h

    def encode(self, x, out, scratch, status):
        x = _dev_u8(x, "x")
        _check(lib().hx_session_encode(self._h, x.data_ptr(), x.numel(), out.data_ptr(),
                                       out.numel(), scratch.data_ptr(), self.hist.data_ptr(),
                                       status.data_ptr(), _stream(x)), "hx_session_encode")
        return out

    def decode(self, stream, n: int, out, status, nbytes=None):
        stream = _dev_u8(stream, "stream")
        _check(lib().hx_session_decode(self._h, stream.data_ptr(), int(nbytes or stream.numel()),
                                       out.data_ptr() if n else stream.data_ptr(), n,
                                       status.data_ptr(), _stream(stream)), "hx_session_decode")
        return out

    def drain(self):
        _check(lib().hx_session_drain(self._h), "hx_session_drain")

    def info(self, batch: int) -> dict:
        b = _BatchInfo()
        _check(lib().hx_session_batch_info(self._h, batch, ctypes.byref(b)),
               "hx_session_batch_info")
        return {"hash": int(b.hash), "slot": int(b.slot), "observed": bool(b.observed),
                "refreshed": bool(b.refreshed), "symbols": int(b.symbols),
                "drift": float(b.drift)}

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.hx_session_destroy(h)


# --------------------------------------------------------------------------------- 8-bit rows
# A matrix kept as bytes (uint8, contiguous) and one float32 scale per row (include/hx.h, "8-bit
# rows"). Every call runs on the tensors' device and that device's current stream, whichever device is
# current; outputs are allocated unless they are given. The calls are explicit forward and backward passes: they record
# no autograd graph. A small call's time is its host time, so the
# checks are plain comparisons and the stream is read as the raw handle.
_torch = None


def _load_torch():
    global _torch, _DTYPES, _raw_stream, _current_device
    import torch
    _DTYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _torch = torch
    return torch


def _dtype(t) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"element type {t.dtype} is not float32, float16 or bfloat16")
    return d


def _launch(dev, what, fn, *args):
    """fn(*args, the current stream of device `dev`), with that device current."""
    if _current_device() == dev:
        rc = fn(*args, _raw_stream(dev))
    else:
        with _torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc:
        raise HxError(rc, what)


def _device(t, what) -> int:
    """The index of the CUDA device of the tensor t."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    return t.get_device()


def _refuse(t, what, shape, dtype, dev):
    """Raises what is wrong with a tensor that should have this shape, element type and device."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must have element type {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on another device than the other tensors")
    raise ValueError(f"{what} must be contiguous")


def _same(t, what, shape, dtype, dev):
    """Checks a tensor's device, element type and shape."""
    if not isinstance(t, _torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, what, shape, dtype, dev)


def _dense(t, what, shape, dtype, dev) -> int:
    """Checks a contiguous tensor; its address."""
    if (not isinstance(t, _torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, what, shape, dtype, dev)
    return t.data_ptr()


def _matrix(t, what):
    """(rows, cols, row stride) of a matrix whose rows are contiguous and do not overlap."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{what} must be a matrix")
    rows, cols = shape
    if (stride[1] != 1 and cols > 1 or stride[0] < cols and rows > 1) and rows and cols:
        raise ValueError(f"{what} must be a matrix of contiguous rows that do not overlap")
    return rows, cols, stride[0]


def _status_ptr(status, dev):
    if status is None:
        return None
    if _device(status, "status") != dev or status.dtype is not _torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 status word on the tensors' device")
    return status.data_ptr()


def quantize_rows(x, fmt: int = ROWS_E4M3, out=None, scale=None):
    """hx_quantize_rows: the rows of the matrix x as (bytes uint8[rows, cols], scale float32[rows])."""
    torch = _torch or _load_torch()
    dev = _device(x, "x")
    dt = _dtype(x)
    rows, cols, ld = _matrix(x, "x")
    if out is None:
        out = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
        ob = out.data_ptr()
    else:
        ob = _dense(out, "out", (rows, cols), torch.uint8, dev)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        sp = scale.data_ptr()
    else:
        sp = _dense(scale, "scale", (rows,), torch.float32, dev)
    _launch(dev, "hx_quantize_rows", lib().hx_quantize_rows, fmt, dt, x.data_ptr(), rows, cols, ld, ob, sp)
    return out, scale


def dequantize_rows(data, scale, fmt: int = ROWS_E4M3, dtype=None, out=None):
    """hx_dequantize_rows: the values of 8-bit rows, as `dtype` (default bfloat16) or into the matrix `out`."""
    torch = _torch or _load_torch()
    dev = _device(data, "bytes")
    shape = data.shape
    if len(shape) != 2:
        raise ValueError("bytes must be a matrix")
    db = _dense(data, "bytes", shape, torch.uint8, dev)
    sp = _dense(scale, "scale", shape[:1], torch.float32, dev)
    if out is None:
        out = torch.empty(*shape, dtype=dtype or torch.bfloat16, device=data.device)
        rows, cols = shape
        ld = cols
    else:
        _same(out, "out", shape, dtype or out.dtype, dev)
        rows, cols, ld = _matrix(out, "out")
    _launch(dev, "hx_dequantize_rows", lib().hx_dequantize_rows, fmt, _dtype(out), db, sp, rows, cols, out.data_ptr(), ld)
    return out


def gated_forward(x, fmt: int = ROWS_E4M3, save: bool = True, out=None):
    """hx_gated_forward: silu(gate) * up of x [rows, 2 cols] (gate first). Returns (h, bytes uint8[rows, 2,
    cols], scale float32[rows, 2]); with save=False (h, None, None)."""
    torch = _torch or _load_torch()
    dev = _device(x, "x")
    dt = _dtype(x)
    rows, both, ld = _matrix(x, "x")
    cols = both // 2
    if both % 2:
        raise ValueError("x must have as many gate columns as up columns")
    if out is None:
        out = torch.empty(rows, cols, dtype=x.dtype, device=x.device)
        op = out.data_ptr()
    else:
        op = _dense(out, "out", (rows, cols), x.dtype, dev)
    data = scale = db = sp = None
    if save:
        data = torch.empty(rows, 2, cols, dtype=torch.uint8, device=x.device)
        scale = torch.empty(rows, 2, dtype=torch.float32, device=x.device)
        db, sp = data.data_ptr(), scale.data_ptr()
    _launch(dev, "hx_gated_forward", lib().hx_gated_forward, fmt, dt, x.data_ptr(), rows, cols, ld, op, db, sp)
    return out, data, scale


def gated_backward(dh, data, scale, fmt: int = ROWS_E4M3, need_h: bool = False):
    """hx_gated_backward: (gradient of x [rows, 2 cols], the activation h again or None) for the gradient dh of
    gated_forward's output, at the saved gate and up."""
    torch = _torch or _load_torch()
    dev = _device(dh, "dh")
    dt = _dtype(dh)
    rows, cols, ld = _matrix(dh, "dh")
    db = _dense(data, "bytes", (rows, 2, cols), torch.uint8, dev)
    sp = _dense(scale, "scale", (rows, 2), torch.float32, dev)
    dx = torch.empty(rows, 2 * cols, dtype=dh.dtype, device=dh.device)
    h = torch.empty(rows, cols, dtype=dh.dtype, device=dh.device) if need_h else None
    _launch(dev, "hx_gated_backward", lib().hx_gated_backward, fmt, dt, dh.data_ptr(), ld, db, sp, rows, cols,
            dx.data_ptr(), h.data_ptr() if need_h else None)
    return dx, h


def _heads(t, what):
    """Token and head strides of [tokens, heads, dim] whose heads are contiguous."""
    stride = t.stride()
    if len(stride) != 3 or (stride[2] != 1 and t.shape[2] > 1 and t.numel()):
        raise ValueError(f"{what} must be [tokens, heads, dim] with contiguous heads")
    return stride[0], stride[1]


def _heads_out(t, shape, dtype, dev):
    """As _heads, for an output: two of its heads may not overlap."""
    _same(t, "out", shape, dtype, dev)
    a, b = _heads(t, "out")
    if t.numel():
        # the shorter stride clears a head, the longer one everything under it
        at = sorted((s, n) for s, n in ((a, shape[0]), (b, shape[1])) if n > 1)
        span = shape[2]
        for s, n in at:
            if s < span:
                raise ValueError("out must not overlap itself")
            span = s * (n - 1) + span
    return a, b


# hx_head_norm_rope, field by field
_NORM = struct.Struct("@IIIIQIIIIIfQPPPPP")


def _head_norm_rope(t, dev, dt, q_heads, wq, wk, cos, sin, positions, eps, interleaved, fmt):
    torch = _torch
    tokens, heads, dim = t.shape
    if not 0 <= q_heads <= heads:
        raise ValueError("q_heads must be between 0 and the number of heads")
    w = wk if wq is None else wq
    if w is None or (q_heads and wq is None) or (q_heads < heads and wk is None):
        raise ValueError("a weight is missing")
    _device(w, "a weight")
    wp = 0 if wq is None else _dense(wq, "wq", (dim,), w.dtype, dev)
    kp = 0 if wk is None else _dense(wk, "wk", (dim,), w.dtype, dev)
    _device(cos, "cos")
    table = cos.shape
    if len(table) != 2:
        raise ValueError("cos and sin must be [places, rot_dim / 2]")
    cp = _dense(cos, "cos", table, torch.float32, dev)
    sp = _dense(sin, "sin", table, torch.float32, dev)
    _device(positions, "positions")
    long = positions.dtype is torch.int64
    pp = _dense(positions, "positions", (tokens,), torch.int64 if long else torch.int32, dev)
    return _NORM.pack(fmt, dt, _dtype(w), 64 if long else 32, tokens, q_heads, heads - q_heads, dim, 2 * table[1],
                      1 if interleaved else 0, eps, table[0], wp, kp, cp, sp, pp)


def head_norm_rope_forward(x, q_heads: int, wq, wk, cos, sin, positions, eps: float = 1e-6,
                           interleaved: bool = False, fmt: int = ROWS_E4M3, save: bool = True, out=None,
                           status=None):
    """hx_head_norm_rope_forward: norm of each head of x [tokens, heads, dim] (queries, then keys) and the
    rotation of its first 2 * cos.shape[1] values by row positions[t] of cos and sin. Returns (y, bytes
    uint8[tokens, heads, dim], scale float32[tokens, heads]); with save=False (y, None, None). `out` may
    be x."""
    torch = _torch or _load_torch()
    dev = _device(x, "x")
    dt = _dtype(x)
    xt, xh = _heads(x, "x")
    p = _head_norm_rope(x, dev, dt, q_heads, wq, wk, cos, sin, positions, eps, interleaved, fmt)
    shape = x.shape
    if out is None:
        out = torch.empty(*shape, dtype=x.dtype, device=x.device)
        yt, yh = out.stride()[:2]
    else:
        yt, yh = _heads_out(out, shape, x.dtype, dev)
    data = scale = db = sp = None
    if save:
        data = torch.empty(*shape, dtype=torch.uint8, device=x.device)
        scale = torch.empty(*shape[:2], dtype=torch.float32, device=x.device)
        db, sp = data.data_ptr(), scale.data_ptr()
    _launch(dev, "hx_head_norm_rope_forward", lib().hx_head_norm_rope_forward, p, x.data_ptr(), xt, xh, out.data_ptr(),
            yt, yh, db, sp, _status_ptr(status, dev))
    return out, data, scale


def head_norm_rope_backward(dy, data, scale, q_heads: int, wq, wk, cos, sin, positions, eps: float = 1e-6,
                            interleaved: bool = False, fmt: int = ROWS_E4M3, out=None, status=None):
    """hx_head_norm_rope_backward: (dx, dwq, dwk) at the saved x; the weights' gradients are float32 (None for a
    weight that is None). `out` (dx) may be dy."""
    torch = _torch or _load_torch()
    dev = _device(dy, "dy")
    dt = _dtype(dy)
    gt, gh = _heads(dy, "dy")
    p = _head_norm_rope(dy, dev, dt, q_heads, wq, wk, cos, sin, positions, eps, interleaved, fmt)
    shape = dy.shape
    db = _dense(data, "bytes", shape, torch.uint8, dev)
    sp = _dense(scale, "scale", shape[:2], torch.float32, dev)
    if out is None:
        out = torch.empty(*shape, dtype=dy.dtype, device=dy.device)
        ot, oh = out.stride()[:2]
    else:
        ot, oh = _heads_out(out, shape, dy.dtype, dev)
    dim = shape[2]
    fn = lib()
    need = fn.hx_head_norm_rope_workspace(dim)
    ws = torch.empty(need, dtype=torch.uint8, device=dy.device)
    dwq = torch.empty(dim, dtype=torch.float32, device=dy.device) if wq is not None else None
    dwk = torch.empty(dim, dtype=torch.float32, device=dy.device) if wk is not None else None
    _launch(dev, "hx_head_norm_rope_backward", fn.hx_head_norm_rope_backward, p, dy.data_ptr(), gt, gh, db, sp,
            out.data_ptr(), ot, oh, dwq.data_ptr() if dwq is not None else None,
            dwk.data_ptr() if dwk is not None else None, ws.data_ptr(), need, _status_ptr(status, dev))
    return out, dwq, dwk


def weight_grad(dy, data, scale, fmt: int = ROWS_E4M3, out=None, dtype=None, accumulate: bool = False,
                status=None):
    """hx_weight_grad: dY^T X [n_out, n_in] of a linear layer, from dy [tokens, n_out] (float16 or bfloat16) and the
    8-bit rows of its input X [tokens, n_in]. The result has `dtype` (dy's, or float32), or goes to the
    matrix `out`, onto its old values if `accumulate`. If a wait inside the kernel runs out (2 s; it does not, on a sound
    GPU), that part of the result is NaN, and HX_ERR_TIMEOUT is raised in `status`, if given."""
    torch = _torch or _load_torch()
    dev = _device(dy, "dy")
    dt = _dtype(dy)
    tokens, n_out, ld = _matrix(dy, "dy")
    _device(data, "bytes")
    shape = data.shape
    if len(shape) != 2:
        raise ValueError("bytes must be [tokens, n_in]")
    n_in = shape[1]
    db = _dense(data, "bytes", (tokens, n_in), torch.uint8, dev)
    sp = _dense(scale, "scale", (tokens,), torch.float32, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty(n_out, n_in, dtype=dtype or dy.dtype, device=dy.device)
        ldw, wt = n_in, dt if dtype is None else _dtype(out)
    else:
        _same(out, "out", (n_out, n_in), dtype or out.dtype, dev)
        ldw, wt = _matrix(out, "out")[2], _dtype(out)
    fn = lib()
    yp = dy.data_ptr()
    # rows on 16 (dy) and 8 bytes need no workspace
    need = (fn.hx_weight_grad_workspace(yp, ld, db, tokens, n_out, n_in)
            if (yp | 2 * ld) % 16 or (db | n_in) % 8 else 0)
    ws = torch.empty(need, dtype=torch.uint8, device=dy.device) if need else None
    _launch(dev, "hx_weight_grad", fn.hx_weight_grad, fmt, dt, yp, ld, db, sp, tokens, n_out, n_in, wt,
            out.data_ptr(), ldw, 1 if accumulate else 0, ws.data_ptr() if need else None, need, _status_ptr(status, dev))
    return out


def weight_grad_bounded(dy, data, scale, out, wait_ns: int, withhold: int = (1 << 64) - 1, fmt: int = ROWS_E4M3,
                        accumulate: bool = False, status=None):
    """hx_weight_grad_bounded: weight_grad() into `out` with its waits' limit in nanoseconds and, for failure tests, a
    block of the launch (`withhold`) whose part never counts as ready. Returns (out, status)."""
    torch = _torch or _load_torch()
    dev = _device(dy, "dy")
    tokens, n_out, ld = _matrix(dy, "dy")
    _device(data, "bytes")
    n_in = data.shape[-1]
    db = _dense(data, "bytes", (tokens, n_in), torch.uint8, dev)
    sp = _dense(scale, "scale", (tokens,), torch.float32, dev)
    _same(out, "out", (n_out, n_in), out.dtype, dev)
    if status is None:
        status = new_status(dy.device)
    need = lib().hx_weight_grad_workspace(dy.data_ptr(), ld, db, tokens, n_out, n_in)
    ws = torch.empty(need, dtype=torch.uint8, device=dy.device)
    _launch(dev, "hx_weight_grad_bounded", lib().hx_weight_grad_bounded, fmt, _dtype(dy), dy.data_ptr(), ld, db, sp, tokens,
            n_out, n_in, _dtype(out), out.data_ptr(), _matrix(out, "out")[2], 1 if accumulate else 0, ws.data_ptr(), need,
            _status_ptr(status, dev), wait_ns, withhold)
    return out, status
