"""Thin Python binding of the C ABI in ``include/tq.h`` (libtq.so).

Argument marshalling only: every step of compression and attention runs in the
library's CUDA kernels.  PyTorch provides device memory and streams.  Importing
this module loads libtq.so and raises ImportError when it is missing or fails
to load; there is no fallback path.

Functions keep the C names: ``tq_make_rotation``, ``tq_fit_codebook``,
``tq_make_qjl``, ``tq_packed_size``, ``tq_compress``, ``tq_dequantize``,
``tq_age_tiers``, ``tq_decode_workspace_size``, ``tq_decode_attention``, and
the serving calls ``tq_rope_table``, ``tq_rope``, ``tq_append``, ``tq_read``,
``tq_tree_workspace_size``, ``tq_tree_attention``, and those on pages and drafts
``tq_page_tables``, ``tq_page_release``, ``tq_paged_append``, ``tq_paged_read``,
``tq_paged_workspace_size``, ``tq_paged_attention``, ``tq_verify``.
Errors come back as ``TQError`` carrying the status and its message.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import numpy as np

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libtq.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"libtq.so not found at {_LIB_PATH}; build it with "
        "`python -m rotated_quantized_kv_gb300.build` (needs nvcc)")
try:
    _lib = ctypes.CDLL(_LIB_PATH)
except OSError as e:  # pragma: no cover - depends on the machine
    raise ImportError(f"cannot load {_LIB_PATH}: {e}") from e

LIB_PATH = _LIB_PATH

TQ_MAX_HEADS = 16
TQ_MAX_SEGMENTS = 8
TQ_MAX_HEAD_DIM = 1024
TQ_SEG_PACKED = 0
TQ_SEG_FP16 = 1
TQ_VALUE_LAW_GAUSS = 0
TQ_VALUE_LAW_SPHERE = 1
TQ_QJL_UNBIASED = 0
TQ_QJL_SIGN_PAIR = 1
TQ_ERR_TIMEOUT = -6
TQ_WAIT_POLLS_DEFAULT = 1 << 20

STATUS = {0: "TQ_OK", -1: "TQ_ERR_ARG", -2: "TQ_ERR_UNSUPPORTED", -3: "TQ_ERR_ALIGN",
          -4: "TQ_ERR_SIZE", -5: "TQ_ERR_CUDA", -6: "TQ_ERR_TIMEOUT"}

EXPORTED = ["tq_status_string", "tq_last_cuda_error", "tq_version", "tq_make_rotation",
            "tq_fit_codebook", "tq_make_qjl", "tq_packed_size", "tq_compress", "tq_dequantize",
            "tq_age_tiers", "tq_decode_workspace_size", "tq_decode_attention",
            "tq_set_decode_kernel_events", "tq_decode_attention_static", "tq_decode_error_flag",
            "tq_requantize", "tq_fit_codebook_sphere", "tq_make_haar_rotation", "tq_compress_error_flag", "tq_decode_last_launches",
            "tq_set_decode_wait_polls", "tq_value_code_table", "tq_rope_frequencies", "tq_rope_table", "tq_rope",
            "tq_append", "tq_read", "tq_tree_workspace_size", "tq_tree_attention", "tq_page_tables", "tq_page_release",
            "tq_paged_append", "tq_paged_read", "tq_paged_workspace_size", "tq_paged_attention", "tq_verify"]

TQ_DTYPE_F16, TQ_DTYPE_BF16, TQ_DTYPE_F32 = 0, 1, 2
TQ_ROPE_SCALE_NONE, TQ_ROPE_SCALE_LINEAR, TQ_ROPE_SCALE_BASE, TQ_ROPE_SCALE_TURNS, TQ_ROPE_SCALE_INDEX = range(5)
TQ_ROPE_HALF, TQ_ROPE_INTERLEAVED = 0, 1
TQ_MAX_ROPE_TENSORS = 4
TQ_MAX_DRAFTS = 256


class TQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.tq_status_string(status).decode()
        if status == -5:
            msg += f" (cudaError {_lib.tq_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")


class tq_rotation(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("seed", ctypes.c_uint64),
                ("sign_bits", ctypes.c_uint32 * (TQ_MAX_HEAD_DIM // 32)), ("dense", ctypes.c_void_p)]


class tq_segment_layout(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("capacity", ctypes.c_int), ("jl_dim", ctypes.c_int),
                ("kbits", ctypes.c_uint8 * TQ_MAX_HEADS), ("vbits", ctypes.c_uint8 * TQ_MAX_HEADS),
                ("qjl", ctypes.c_uint8 * TQ_MAX_HEADS), ("value_law", ctypes.c_uint8),
                ("qjl_v", ctypes.c_uint8 * TQ_MAX_HEADS)]


class tq_packed_sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("kcode_bytes", "vcode_bytes", "kscale_bytes",
                                                "vscale_bytes", "qjl_sign_bytes", "qjl_norm_bytes",
                                                "vqjl_sign_bytes", "vqjl_norm_bytes")]


class tq_packed_bufs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("kcodes", "vcodes", "kscale", "vscale",
                                                "qjl_signs", "qjl_norm", "vqjl_signs", "vqjl_norm")]


class tq_segment(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("n_tokens", ctypes.c_int), ("layout", tq_segment_layout),
                ("packed", tq_packed_bufs), ("k16", ctypes.c_void_p), ("v16", ctypes.c_void_p),
                ("attn_mass", ctypes.c_void_p)]


class tq_layer_view(ctypes.Structure):
    _fields_ = [("rot", tq_rotation), ("n_segments", ctypes.c_int),
                ("seg", tq_segment * TQ_MAX_SEGMENTS), ("qjl_estimator", ctypes.c_int)]


class tq_rope_spec(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("scaling", ctypes.c_int)] + [
        (n, ctypes.c_double) for n in ("base", "factor", "original_len", "fast", "slow", "amplitude")]


class tq_rope_view(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int), ("n_pos", ctypes.c_int),
                ("table", ctypes.c_void_p)]


class tq_rope_tensor(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n_heads", ctypes.c_int),
                ("in_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


class tq_tree(ctypes.Structure):
    _fields_ = [("n_drafts", ctypes.c_int), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("mask", ctypes.c_void_p), ("mask_stride_b", ctypes.c_int64),
                ("seg_len", ctypes.c_void_p * TQ_MAX_SEGMENTS), ("out", ctypes.c_void_p)]


class tq_pages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride_b", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("len", ctypes.c_void_p)]


class tq_verification(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "n_drafts", "vocab", "dtype")] + [
        ("tokens", ctypes.c_void_p), ("tokens_stride_b", ctypes.c_int64), ("parents", ctypes.c_void_p),
        ("parents_stride_b", ctypes.c_int64), ("target", ctypes.c_void_p), ("target_stride", ctypes.c_int64 * 2),
        ("draft", ctypes.c_void_p), ("draft_stride", ctypes.c_int64 * 2), ("uniform", ctypes.c_void_p),
        ("uniform_stride_b", ctypes.c_int64), ("accepted", ctypes.c_void_p), ("n_accepted", ctypes.c_void_p),
        ("token", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_lib.tq_status_string.restype = ctypes.c_char_p
_lib.tq_status_string.argtypes = [_I]
_lib.tq_last_cuda_error.restype = _I
_lib.tq_version.restype = _I
_lib.tq_decode_last_launches.restype = _I
_lib.tq_decode_last_launches.argtypes = []
_lib.tq_make_rotation.argtypes = [_I, ctypes.c_uint64, ctypes.POINTER(tq_rotation)]
_lib.tq_fit_codebook.argtypes = [_I, _P, _P]
_lib.tq_fit_codebook_sphere.argtypes = [_I, _I, _P, _P]
_lib.tq_value_code_table.argtypes = [_I, _P, _P]
_lib.tq_make_haar_rotation.argtypes = [_I, ctypes.c_uint64, _P]
_lib.tq_compress_error_flag.argtypes = [ctypes.POINTER(ctypes.c_int), _I]
_lib.tq_make_qjl.argtypes = [_I, _I, ctypes.c_uint64, _P]
_lib.tq_packed_size.argtypes = [ctypes.POINTER(tq_segment_layout), ctypes.POINTER(tq_packed_sizes)]
_lib.tq_compress.argtypes = [ctypes.POINTER(tq_segment_layout), ctypes.POINTER(tq_rotation), _P, _P, _P,
                             _I, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _I,
                             ctypes.POINTER(tq_packed_bufs), _P]
_lib.tq_dequantize.argtypes = [ctypes.POINTER(tq_segment_layout), ctypes.POINTER(tq_packed_bufs),
                               ctypes.POINTER(tq_rotation), _I, _I, _P, _P, _P, _P, _P]
_lib.tq_requantize.argtypes = [ctypes.POINTER(tq_segment_layout), ctypes.POINTER(tq_packed_bufs), _I,
                               ctypes.POINTER(tq_segment_layout), ctypes.POINTER(tq_packed_bufs), _I, _I, _P]
_lib.tq_age_tiers.argtypes = [_I, _I, _P, _P, _P]
_lib.tq_decode_workspace_size.argtypes = [ctypes.POINTER(tq_layer_view), _I, _I, _I, _I, _I,
                                          ctypes.POINTER(ctypes.c_size_t)]
_lib.tq_decode_attention.argtypes = [ctypes.POINTER(tq_layer_view), _I, _I, _I, _I, _I, _P, _I, _P, _P,
                                     _P, ctypes.c_size_t, _P]
_lib.tq_set_decode_kernel_events.argtypes = [_P, _P]
_lib.tq_decode_error_flag.argtypes = [_P, ctypes.POINTER(ctypes.c_int), _P]
_lib.tq_set_decode_wait_polls.argtypes = [_I]
_lib.tq_decode_attention_static.argtypes = [ctypes.POINTER(tq_layer_view), _I, _I, _I, _I, _I, _P, _I, _P,
                                            _P, _P]
_lib.tq_rope_frequencies.argtypes = [ctypes.POINTER(tq_rope_spec), _P]
_lib.tq_rope_table.argtypes = [ctypes.POINTER(tq_rope_spec), _I, _I, _P, _P]
_lib.tq_rope.argtypes = [ctypes.POINTER(tq_rope_view), _I, _I, _I, _I, _P, _L, _P, _I, _I,
                         _P]
_lib.tq_append.argtypes = [_P, ctypes.POINTER(tq_rotation), ctypes.POINTER(tq_rope_view), _P, _L,
                           _P, _P, _P, _P, _I, _I, _P, _P, _P, _L, _P]
_lib.tq_read.argtypes = [_P, ctypes.POINTER(tq_rotation), _I, _P, _P, _I, _P, _P, _P, _P, _P]
_lib.tq_tree_workspace_size.argtypes = [ctypes.POINTER(tq_layer_view), _I, _I, _I, _I, _I,
                                        ctypes.POINTER(ctypes.c_size_t)]
_lib.tq_tree_attention.argtypes = [ctypes.POINTER(tq_layer_view), _I, _I, _I, _I, _P, _P,
                                   ctypes.c_size_t, _P]
_lib.tq_page_tables.argtypes = [_I, _I, _I, _I, _P, _L, _P, _P, _I, _P, _P, _P, _P, _P, _P]
_lib.tq_page_release.argtypes = [_I, _I, _I, _I, _P, _L, _P, _P, _P, _P, _P]
_lib.tq_paged_append.argtypes = [_P, ctypes.POINTER(tq_rotation), ctypes.POINTER(tq_rope_view), _P, _L,
                                 _P, _P, _P, _P, _I, _I, _I, _P, _L, _P, _P, _L, _P]
_lib.tq_paged_read.argtypes = [_P, ctypes.POINTER(tq_rotation), _I, _I, _P, _L, _P, _I, _P, _P, _P, _P, _P]
_lib.tq_paged_workspace_size.argtypes = [ctypes.POINTER(tq_layer_view), _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]
_lib.tq_paged_attention.argtypes = [ctypes.POINTER(tq_layer_view), _P, _I, _I, _I, _I, _P, _P, _P, _P,
                                    ctypes.c_size_t, _P]
_lib.tq_verify.argtypes = [_P, _P]
TQ_STATIC_WORKSPACE_BYTES = 16 << 20
for _n in EXPORTED:
    if _n not in ("tq_status_string", "tq_last_cuda_error", "tq_version", "tq_decode_last_launches"):
        getattr(_lib, _n).restype = _I


def _check(status: int, where: str):
    if status != 0:
        raise TQError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def on_stream(stream, device):
    """Context in which torch's own work goes to `stream` (a torch stream, a raw handle of one of `device`, or
    None: the current one), as what a call prepares has to go where its kernels run."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        raw = int(stream)
        stream = torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


# ----------------------------------------------------------------- host calls
def tq_version() -> int:
    return _lib.tq_version()


def tq_make_rotation(head_dim: int, seed: int) -> tq_rotation:
    rot = tq_rotation()
    _check(_lib.tq_make_rotation(head_dim, seed, ctypes.byref(rot)), "tq_make_rotation")
    return rot


def tq_fit_codebook(bits: int):
    """(centroids, thresholds) as float32 CPU tensors."""
    c = torch.zeros(1 << bits, dtype=torch.float32)
    t = torch.zeros(max((1 << bits) - 1, 1), dtype=torch.float32)
    _check(_lib.tq_fit_codebook(bits, c.data_ptr(), t.data_ptr()), "tq_fit_codebook")
    return c, t[: (1 << bits) - 1]


def tq_value_code_table(bits: int, thresholds) -> np.ndarray:
    """The compressor's value-code lookup table (2048 uint32) for 1-4 bits and
    an ascending binary32 threshold set (see include/tq.h)."""
    t = np.ascontiguousarray(np.asarray(thresholds, dtype=np.float32))
    out = np.zeros(2048, dtype=np.uint32)
    _check(_lib.tq_value_code_table(bits, t.ctypes.data, out.ctypes.data), "tq_value_code_table")
    return out


def tq_fit_codebook_sphere(bits: int, head_dim: int = 128):
    """(centroids, thresholds) of the sphere-coordinate law, float32 CPU tensors."""
    c = torch.zeros(1 << bits, dtype=torch.float32)
    t = torch.zeros(max((1 << bits) - 1, 1), dtype=torch.float32)
    _check(_lib.tq_fit_codebook_sphere(bits, head_dim, c.data_ptr(), t.data_ptr()), "tq_fit_codebook_sphere")
    return c, t[: (1 << bits) - 1]


def tq_make_haar_rotation(head_dim: int, seed: int) -> torch.Tensor:
    """Haar-random rotation Q (float32 CPU tensor [d][d], y = Q x)."""
    Q = torch.zeros(head_dim, head_dim, dtype=torch.float32)
    _check(_lib.tq_make_haar_rotation(head_dim, seed, Q.data_ptr()), "tq_make_haar_rotation")
    return Q


def dense_rotation(rot: tq_rotation, Q: torch.Tensor) -> tq_rotation:
    """A copy of ``rot`` that rotates with the dense matrix Q (a float32 CUDA
    tensor [d][d] the caller keeps alive) instead of the SRHT."""
    r = tq_rotation()
    ctypes.pointer(r)[0] = rot
    assert Q.dtype == torch.float32 and Q.is_contiguous() and tuple(Q.shape) == (rot.head_dim, rot.head_dim)
    r.dense = Q.data_ptr()
    return r


def tq_compress_error_flag(reset: bool = False) -> int:
    """The dense compressor's timeout flag (0: none); the call's TQ_ERR_TIMEOUT
    status is returned as the flag, not raised."""
    f = ctypes.c_int(0)
    st = _lib.tq_compress_error_flag(ctypes.byref(f), int(reset))
    if st != TQ_ERR_TIMEOUT:
        _check(st, "tq_compress_error_flag")
    return f.value


def tq_make_qjl(head_dim: int, jl_dim: int, seed: int) -> torch.Tensor:
    """QJL projection S (float32 CPU tensor [jl_dim][head_dim])."""
    S = torch.zeros(jl_dim, head_dim, dtype=torch.float32)
    _check(_lib.tq_make_qjl(head_dim, jl_dim, seed, S.data_ptr()), "tq_make_qjl")
    return S


def make_layout(batch, n_heads, head_dim, capacity, kbits, vbits, qjl=None, jl_dim=128, value_law=0, qjl_v=None):
    L = tq_segment_layout()
    L.batch, L.n_heads, L.head_dim, L.capacity, L.jl_dim = batch, n_heads, head_dim, capacity, jl_dim
    L.value_law = value_law
    kb = [int(kbits)] * n_heads if isinstance(kbits, int) else [int(x) for x in kbits]
    vb = [int(vbits)] * n_heads if isinstance(vbits, int) else [int(x) for x in vbits]
    qj = [0] * n_heads if qjl is None else [int(bool(x)) for x in qjl]
    qv = [0] * n_heads if qjl_v is None else [int(bool(x)) for x in qjl_v]
    for h in range(n_heads):
        L.kbits[h], L.vbits[h], L.qjl[h], L.qjl_v[h] = kb[h], vb[h], qj[h], qv[h]
    return L


def tq_packed_size(layout: tq_segment_layout) -> tq_packed_sizes:
    s = tq_packed_sizes()
    _check(_lib.tq_packed_size(ctypes.byref(layout), ctypes.byref(s)), "tq_packed_size")
    return s


def tq_age_tiers(n_tokens: int, age_bounds):
    b = (ctypes.c_int * max(len(age_bounds), 1))(*age_bounds)
    start = (ctypes.c_int * (len(age_bounds) + 1))()
    end = (ctypes.c_int * (len(age_bounds) + 1))()
    _check(_lib.tq_age_tiers(n_tokens, len(age_bounds), b, start, end), "tq_age_tiers")
    return list(zip(start, end))


# ----------------------------------------------------------------- segments
_pack_segment = struct.Struct(f"ii{ctypes.sizeof(tq_segment_layout)}s8PPPP").pack
assert struct.calcsize(f"ii{ctypes.sizeof(tq_segment_layout)}s8PPPP") == ctypes.sizeof(tq_segment)


class PackedSegment:
    """Device buffers of one packed segment, allocated with torch from the sizes
    tq_packed_size reports."""

    kind = TQ_SEG_PACKED
    attn_mass = None  # optional float tensor [B][H][capacity]: written by tq_decode_attention

    def __init__(self, layout: tq_segment_layout, device="cuda", n_tokens: int = 0):
        self.layout = layout
        self.n_tokens = n_tokens
        s = tq_packed_size(layout)
        u8 = dict(dtype=torch.uint8, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.kcodes = torch.zeros(max(s.kcode_bytes, 16), **u8)
        self.vcodes = torch.zeros(max(s.vcode_bytes, 16), **u8)
        self.kscale = torch.zeros(max(s.kscale_bytes // 4, 4), **f32)
        self.vscale = torch.zeros(max(s.vscale_bytes // 4, 4), **f32)
        self.qjl_signs = torch.zeros(max(s.qjl_sign_bytes, 16), **u8) if s.qjl_sign_bytes else None
        self.qjl_norm = torch.zeros(max(s.qjl_norm_bytes // 4, 4), **f32) if s.qjl_norm_bytes else None
        self.vqjl_signs = torch.zeros(max(s.vqjl_sign_bytes, 16), **u8) if s.vqjl_sign_bytes else None
        self.vqjl_norm = torch.zeros(max(s.vqjl_norm_bytes // 4, 4), **f32) if s.vqjl_norm_bytes else None

    def bufs(self) -> tq_packed_bufs:
        b = tq_packed_bufs()
        b.kcodes, b.vcodes = _ptr(self.kcodes), _ptr(self.vcodes)
        b.kscale, b.vscale = _ptr(self.kscale), _ptr(self.vscale)
        b.qjl_signs, b.qjl_norm = _ptr(self.qjl_signs), _ptr(self.qjl_norm)
        b.vqjl_signs, b.vqjl_norm = _ptr(self.vqjl_signs), _ptr(self.vqjl_norm)
        return b

    def segment(self) -> tq_segment:
        s = tq_segment()
        s.kind, s.n_tokens, s.layout, s.packed = TQ_SEG_PACKED, self.n_tokens, self.layout, self.bufs()
        s.attn_mass = _ptr(self.attn_mass)
        return s

    def reference(self) -> bytes:
        """The segment as a serving call is handed it: a tq_segment of its own each time, the fields that these
        calls read (no sketches, no attn_mass)."""
        return _pack_segment(TQ_SEG_PACKED, self.n_tokens, bytes(self.layout), self.kcodes.data_ptr(), self.vcodes.data_ptr(),
                             self.kscale.data_ptr(), self.vscale.data_ptr(), 0, 0, 0, 0, 0, 0, 0)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.kcodes, self.vcodes, self.kscale, self.vscale, self.qjl_signs, self.qjl_norm,
                    self.vqjl_signs, self.vqjl_norm)
                   if t is not None)


class Fp16Segment:
    """Tokens kept verbatim in fp16: [B][H][capacity][d] K and V."""

    kind = TQ_SEG_FP16
    attn_mass = None  # optional float tensor [B][H][capacity]: written by tq_decode_attention

    def __init__(self, batch, n_heads, head_dim, capacity, device="cuda", n_tokens=0, k=None, v=None):
        self.layout = make_layout(batch, n_heads, head_dim, capacity, 1, 1)
        self.n_tokens = n_tokens
        shape = (batch, n_heads, capacity, head_dim)
        self.k = k if k is not None else torch.zeros(shape, dtype=torch.float16, device=device)
        self.v = v if v is not None else torch.zeros(shape, dtype=torch.float16, device=device)

    def segment(self) -> tq_segment:
        s = tq_segment()
        s.kind, s.n_tokens, s.layout = TQ_SEG_FP16, self.n_tokens, self.layout
        s.k16, s.v16 = _ptr(self.k), _ptr(self.v)
        s.attn_mass = _ptr(self.attn_mass)
        return s

    def reference(self) -> bytes:
        """The segment as a serving call is handed it (see PackedSegment.reference)."""
        return _pack_segment(TQ_SEG_FP16, self.n_tokens, bytes(self.layout), 0, 0, 0, 0, 0, 0, 0, 0, self.k.data_ptr(),
                             self.v.data_ptr(), 0)


def layer_view(rot: tq_rotation, segments, qjl_estimator: int = TQ_QJL_UNBIASED) -> tq_layer_view:
    """A layer's segments; a segment's attn_mass tensor (if set) receives the
    attention mass of its tokens at the next decode call."""
    lv = tq_layer_view()
    lv.rot = rot
    lv.qjl_estimator = qjl_estimator
    lv.n_segments = len(segments)
    for i, s in enumerate(segments):
        lv.seg[i] = s.segment()
    return lv


# ----------------------------------------------------------------- device calls
def tq_compress(seg: PackedSegment, rot: tq_rotation, K: torch.Tensor, V: torch.Tensor, t_begin: int = 0,
                qjl_S: torch.Tensor | None = None, stream=None):
    """Compress K, V (fp16 CUDA tensors [B][H][T][d], unit stride in d) into
    positions [t_begin, t_begin + T) of ``seg``."""
    B, H, T, d = K.shape
    assert V.shape == K.shape and V.stride() == K.stride() and K.dtype == torch.float16
    sb, sh, st, si = K.stride()
    assert si == 1
    _check(_lib.tq_compress(ctypes.byref(seg.layout), ctypes.byref(rot), _ptr(qjl_S), _ptr(K), _ptr(V), T,
                            sb, sh, st, t_begin, ctypes.byref(seg.bufs()), _stream(stream)), "tq_compress")
    seg.n_tokens = max(seg.n_tokens, t_begin + T)


def tq_requantize(src: PackedSegment, src_t_begin: int, n_tokens: int, dst: PackedSegment, dst_t_begin: int,
                  stream=None):
    """Tier demotion: tokens [src_t_begin, src_t_begin + n) of src re-quantised
    in the rotated space with dst's widths into [dst_t_begin, dst_t_begin + n)."""
    _check(_lib.tq_requantize(ctypes.byref(src.layout), ctypes.byref(src.bufs()), src_t_begin,
                              ctypes.byref(dst.layout), ctypes.byref(dst.bufs()), dst_t_begin, n_tokens,
                              _stream(stream)), "tq_requantize")
    dst.n_tokens = max(dst.n_tokens, dst_t_begin + n_tokens)


def tq_dequantize(seg: PackedSegment, t_begin: int, n_tokens: int, rot: tq_rotation | None = None,
                  rotated: bool = True, original: bool = False, stream=None):
    """(k_rot, v_rot, k_orig, v_orig) float32 [B][H][n][d] CUDA tensors (None where not asked), allocated
    for `stream`."""
    L = seg.layout
    shape = (L.batch, L.n_heads, n_tokens, L.head_dim)
    dev = seg.kcodes.device
    mk = (lambda: torch.empty(shape, dtype=torch.float32, device=dev))
    with on_stream(stream, dev):
        kr, vr = (mk(), mk()) if rotated else (None, None)
        ko, vo = (mk(), mk()) if original else (None, None)
    _check(_lib.tq_dequantize(ctypes.byref(L), ctypes.byref(seg.bufs()),
                              ctypes.byref(rot) if rot is not None else None, t_begin, n_tokens,
                              _ptr(kr), _ptr(vr), _ptr(ko), _ptr(vo), _stream(stream)), "tq_dequantize")
    return kr, vr, ko, vo


def _views(layers):
    arr = (tq_layer_view * len(layers))()
    for i, lv in enumerate(layers):
        arr[i] = lv
    return arr


def tq_decode_workspace_size(layers, batch, n_heads, q_heads, head_dim) -> int:
    n = ctypes.c_size_t()
    _check(_lib.tq_decode_workspace_size(_views(layers), len(layers), batch, n_heads, q_heads, head_dim,
                                         ctypes.byref(n)), "tq_decode_workspace_size")
    return n.value


def tq_decode_attention(layers, q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                        n_heads: int, qjl_S: torch.Tensor | None = None, jl_dim: int = 128, stream=None,
                        views=None):
    """out[l][b][j] = attention of q[l][b][j] (fp16) over layer l's segments.
    ``layers`` is a list of tq_layer_view; ``views`` may pass a prebuilt ctypes array."""
    L, B, Hq, d = q.shape
    arr = views if views is not None else _views(layers)
    _check(_lib.tq_decode_attention(arr, L, B, n_heads, Hq, d, _ptr(qjl_S), jl_dim, _ptr(q), _ptr(out),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "tq_decode_attention")
    return out


def tq_decode_last_launches() -> int:
    """Kernel launches this thread's last decode call made."""
    return _lib.tq_decode_last_launches()


def tq_set_decode_kernel_events(start=None, stop=None):
    """Time the packed split-K kernel alone: pass two torch.cuda.Event objects
    (created with enable_timing=True), or None, None to stop."""
    sp = start.cuda_event if start is not None else None
    ep = stop.cuda_event if stop is not None else None
    _check(_lib.tq_set_decode_kernel_events(sp, ep), "tq_set_decode_kernel_events")


def tq_decode_attention_static(layers, q: torch.Tensor, out: torch.Tensor, n_heads: int,
                               qjl_S: torch.Tensor | None = None, jl_dim: int = 128, stream=None, views=None):
    """tq_decode_attention without a workspace argument: the library's fixed
    TQ_STATIC_WORKSPACE_BYTES device array is the scratch, so the call allocates
    nothing (for callers that may not allocate device memory while running).
    Calls share that array: keep them ordered on one stream."""
    L, B, Hq, d = q.shape
    arr = views if views is not None else _views(layers)
    _check(_lib.tq_decode_attention_static(arr, L, B, n_heads, Hq, d, _ptr(qjl_S), jl_dim, _ptr(q), _ptr(out),
                                           _stream(stream)), "tq_decode_attention_static")
    return out


def tq_decode_error_flag(workspace: torch.Tensor | None, stream=None) -> int:
    """Non-zero if a decode call on this workspace stopped a CTA after a bounded
    wait for its own copies (never expected); synchronises the stream.  None:
    the static scratch array of tq_decode_attention_static.  The call's
    TQ_ERR_TIMEOUT status is returned as the flag, not raised."""
    f = ctypes.c_int()
    st = _lib.tq_decode_error_flag(_ptr(workspace), ctypes.byref(f), _stream(stream))
    if st != TQ_ERR_TIMEOUT:
        _check(st, "tq_decode_error_flag")
    return f.value


def tq_set_decode_wait_polls(polls: int):
    """Failure-path hook for tests: polls of a split-K CTA's wait for its own
    copies before it gives up (default 2^20; 0 = give up at once)."""
    _check(_lib.tq_set_decode_wait_polls(polls), "tq_set_decode_wait_polls")


def views_array(layers):
    """Prebuilt ctypes array of layer views (reuse across calls to skip marshalling)."""
    return _views(layers)


# ----------------------------------------------------------------- serving
# These calls run once a layer and token, so their marshalling is kept short: structures
# and stride triples are packed in one go, devices compared as numbers, the stream
# taken raw.
_DTYPE = {torch.float16: TQ_DTYPE_F16, torch.bfloat16: TQ_DTYPE_BF16, torch.float32: TQ_DTYPE_F32}
_F16, _I32 = torch.float16, torch.int32
_pack3 = struct.Struct("3q").pack
_pack_rope = [struct.Struct("PPi4x6q" * n).pack for n in range(TQ_MAX_ROPE_TENSORS + 1)]
_pack_tree = struct.Struct(f"i4xPPP9qPq{TQ_MAX_SEGMENTS}PP").pack
assert struct.calcsize("PPi4x6q") == ctypes.sizeof(tq_rope_tensor)
assert struct.calcsize(f"i4xPPP9qPq{TQ_MAX_SEGMENTS}PP") == ctypes.sizeof(tq_tree)


def _require(ok: bool, where: str):
    if not ok:
        raise TQError(-1, where)


def _int32(t, where, shape):
    """Checks an int32 tensor of `shape` with unit stride in its last axis."""
    _require(t.dtype == _I32 and t.shape == shape and (shape[-1] <= 1 or t.stride(-1) == 1), where)


def _call(tensors, stream, where, fn, *args):
    """fn(*args, stream) with the tensors' device current (the library works on the
    current device), on the given stream or that device's current one.  All tensors
    (None: not given) have to be on one CUDA device."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise TQError(-1, where)
    if dev < 0:
        raise TQError(-1, where)
    if stream is not None:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    else:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != 0:
        raise TQError(status, where)


def tq_make_rope(rotary_dim: int, base: float = 10000.0, scaling: int = TQ_ROPE_SCALE_NONE, factor: float = 1.0,
                 original_len: float = 0.0, fast: float = 0.0, slow: float = 0.0,
                 amplitude: float = 1.0) -> tq_rope_spec:
    """Frequencies of rotary positions (see include/tq.h for the scalings)."""
    s = tq_rope_spec(rotary_dim, scaling, base, factor, original_len, fast, slow, amplitude)
    tq_rope_frequencies(s)  # argument errors here
    return s


def tq_rope_frequencies(spec: tq_rope_spec) -> np.ndarray:
    """The pairs' frequencies, binary64."""
    out = np.zeros(max(spec.rotary_dim // 2, 1))
    _check(_lib.tq_rope_frequencies(ctypes.byref(spec), out.ctypes.data), "tq_rope_frequencies")
    return out


def tq_rope_table(spec: tq_rope_spec, n_pos: int, first_pos: int = 0, device="cuda", stream=None) -> torch.Tensor:
    """float32 CUDA table [n_pos][2][rotary_dim / 2] of cosines and sines, allocated for `stream`."""
    _require(n_pos >= 0, "tq_rope_table")
    with on_stream(stream, device):
        t = torch.empty(n_pos, 2, spec.rotary_dim // 2, dtype=torch.float32, device=device)
    _call([t], stream, "tq_rope_table", _lib.tq_rope_table, ctypes.byref(spec), first_pos, n_pos, t.data_ptr())
    return t


class Rope:
    """A table of cosines and sines [n_pos][2][rotary_dim / 2] (float32 CUDA,
    contiguous; tq_rope_table or the caller's own) and the layout of the pairs."""

    def __init__(self, table: torch.Tensor, layout: int = TQ_ROPE_HALF):
        _require(table.dtype == torch.float32 and table.dim() == 3 and table.shape[1] == 2 and table.is_contiguous(),
                 "Rope")
        _require(layout in (TQ_ROPE_HALF, TQ_ROPE_INTERLEAVED), "Rope")
        self.table, self.layout = table, layout
        self.view = tq_rope_view(2 * table.shape[2], layout, table.shape[0], _ptr(table))
        self.ref = ctypes.byref(self.view)


def tq_rope(rope: Rope, positions: torch.Tensor, x, out=None, inverse: bool = False, stream=None):
    """Rotary positions of x (a CUDA tensor [B][H][T][d] of any strides with unit
    stride in d, or a list of up to four of the same B, T, d and type: queries
    and keys) into `out` (likewise; None: in place).  positions: int32 [B][T] or
    [T].  inverse: the transpose (the gradient of x)."""
    one = isinstance(x, torch.Tensor)
    xs = [x] if one else list(x)
    outs = xs if out is None else ([out] if isinstance(out, torch.Tensor) else list(out))
    where = "tq_rope"
    n = len(xs)
    _require(1 <= n <= TQ_MAX_ROPE_TENSORS and n == len(outs) and xs[0].dim() == 4, where)
    dtype = xs[0].dtype
    B, _, T, d = xs[0].shape
    _require(dtype in _DTYPE, where)
    fields = []
    for i, o in zip(xs, outs):
        shape, a, b = i.shape, i.stride(), o.stride()
        _require(len(shape) == 4 and shape == o.shape and shape[0] == B and shape[2] == T and shape[3] == d and
                 i.dtype == dtype and o.dtype == dtype and (d == 1 or a[3] == b[3] == 1), where)
        fields += (i.data_ptr(), o.data_ptr(), shape[1], a[0], a[1], a[2], b[0], b[1], b[2])
    if positions.dim() == 1:
        _int32(positions, where, (T,))
        ps = 0
    else:
        _int32(positions, where, (B, T))
        ps = positions.stride(0)
    _call([positions, rope.table, *xs, *outs], stream, where, _lib.tq_rope, rope.ref, _DTYPE[dtype], B, T, d,
          positions.data_ptr(), ps, _pack_rope[n](*fields), n, 1 if inverse else 0)
    return outs[0] if one else outs


def tq_append(seg, rot: tq_rotation | None, K: torch.Tensor, V: torch.Tensor, t_begin: torch.Tensor, n_new=None,
              index=None, n_max: int | None = None, rope: Rope | None = None, positions=None, stream=None):
    """Write rows of K, V (fp16 CUDA [B][H][S][d], unit stride in d) into `seg`
    (PackedSegment or Fp16Segment) at each sequence's own position: row j <
    min(n_new[b], n_max) of sequence b is source row index[b][j] (None: j) and
    goes to position t_begin[b] + j.  t_begin, n_new: int32 [B]; index: int32
    [B][n_max]; n_max: default the index's width, else S.  rope: rotates the keys
    by positions (int32 [B][S] or [S]) first.  Rows outside the source or the
    segment are skipped.  seg.n_tokens is left to the caller."""
    where = "tq_append"
    L = seg.layout
    shape = K.shape
    _require(len(shape) == 4 and shape == V.shape and K.dtype == _F16 and V.dtype == _F16 and
             shape[0] == L.batch and shape[1] == L.n_heads and shape[3] == L.head_dim, where)
    a, b = K.stride(), V.stride()
    B, S = shape[0], shape[2]
    _require(a[3] == 1 and b[3] == 1, where)
    if n_max is None:
        n_max = index.shape[1] if index is not None else S
    tensors = [K, V, t_begin, seg.kcodes if seg.kind == TQ_SEG_PACKED else seg.k]
    _int32(t_begin, where, (B,))
    n_ptr = index_ptr = pos_ptr = rope_ref = None
    index_stride = ps = 0
    if n_new is not None:
        _int32(n_new, where, (B,))
        n_ptr = n_new.data_ptr()
        tensors.append(n_new)
    if index is not None:
        _require(index.dim() == 2 and index.shape[1] >= n_max, where)
        _int32(index, where, (B, index.shape[1]))
        index_ptr, index_stride = index.data_ptr(), index.stride(0)
        tensors.append(index)
    if rope is not None:
        _require(positions is not None, where)
        _int32(positions, where, (S,) if positions.dim() == 1 else (B, S))
        ps = positions.stride(0) if positions.dim() == 2 else 0
        pos_ptr, rope_ref = positions.data_ptr(), rope.ref
        tensors += (positions, rope.table)
    _call(tensors, stream, where, _lib.tq_append, seg.reference(), ctypes.byref(rot) if rot is not None else None,
          rope_ref, pos_ptr, ps, K.data_ptr(), _pack3(a[0], a[1], a[2]), V.data_ptr(), _pack3(b[0], b[1], b[2]), S, n_max,
          t_begin.data_ptr(), n_ptr, index_ptr, index_stride)


def tq_read(seg, rot: tq_rotation | None, t_begin: torch.Tensor, n_max: int, n_read=None, out=None,
            dtype=torch.float16, stream=None):
    """Rows of `seg` (PackedSegment or Fp16Segment) back as vectors: row j <
    min(n_read[b], n_max) of sequence b is position t_begin[b] + j (int32 [B]
    tensors).  out: [k, v] tensors [B][H][n_max][d] of fp16, bf16 or fp32 (any
    strides with unit stride in d, None entries: not wanted), default new ones of
    `dtype` on `stream`, zero where nothing is read.  rot None: rotated-space vectors."""
    where = "tq_read"
    L = seg.layout
    shape = (L.batch, L.n_heads, n_max, L.head_dim)
    own = seg.kcodes if seg.kind == TQ_SEG_PACKED else seg.k
    if out is None:
        _require(n_max >= 0 and own.is_cuda, where)
        with on_stream(stream, own.device):  # behind this the kernel writes them
            out = [torch.zeros(shape, dtype=dtype, device=own.device) for _ in range(2)]
    k, v = out
    some = [t for t in (k, v) if t is not None]
    _int32(t_begin, where, (L.batch,))
    tensors = [t_begin, own, *some]
    n_ptr = None
    if n_read is not None:
        _int32(n_read, where, (L.batch,))
        n_ptr = n_read.data_ptr()
        tensors.append(n_read)
    if not some:
        return out
    dt = some[0].dtype
    _require(dt in _DTYPE, where)
    args = []
    for t in (k, v):
        if t is None:
            args += (None, None)
            continue
        a = t.stride()
        _require(t.shape == shape and t.dtype == dt and a[3] == 1, where)
        args += (t.data_ptr(), _pack3(a[0], a[1], a[2]))
    _call(tensors, stream, where, _lib.tq_read, seg.reference(), ctypes.byref(rot) if rot is not None else None, n_max,
          t_begin.data_ptr(), n_ptr, _DTYPE[dt], *args)
    return out


def tree_mask(parents: torch.Tensor) -> torch.Tensor:
    """Visibility words of draft trees: parents int [B][N] (or [N]), the index of
    each draft's parent (before it) or -1 at a root; a draft sees itself and its
    ancestors.  int32 [B][N][ceil(N / 32)] (or without B), as tq_tree_attention
    takes it, on the parents' device.  A parent that is not before its draft is none."""
    p = parents if parents.dim() == 2 else parents[None]
    B, N = p.shape
    W = -(-N // 32)
    i = torch.arange(N, device=p.device)
    p = torch.where((p >= 0) & (p < i), p.long(), -1)  # (they index below)
    see = torch.zeros(B, N, W * 32, dtype=torch.bool, device=p.device)
    at = i.expand(B, N).long()
    for _ in range(N):  # one generation a step
        see.scatter_(2, at.clamp(min=0)[..., None], (at >= 0)[..., None] | see.gather(2, at.clamp(min=0)[..., None]))
        at = torch.where(at >= 0, p.gather(1, at.clamp(min=0)), at)
    w = (see.view(B, N, W, 32).long() << torch.arange(32, device=p.device)).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).int()
    return w if parents.dim() == 2 else w[0]


def tq_tree_workspace_size(view: tq_layer_view, batch: int, n_heads: int, q_heads: int, n_drafts: int,
                           head_dim: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.tq_tree_workspace_size(ctypes.byref(view), batch, n_heads, q_heads, head_dim, n_drafts,
                                       ctypes.byref(n)), "tq_tree_workspace_size")
    return n.value


def tq_tree_attention(view: tq_layer_view, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                      workspace: torch.Tensor, mask: torch.Tensor | None = None, seg_len=None, stream=None):
    """out[b][i][j] = attention of drafted token i, query head j over the cache
    `view` and the drafts it sees.  q fp16 [B][N][Hq][d], k, v fp16 [B][H][N][d]
    (any strides with unit stride in d), out fp16 [B][N][Hq][d] contiguous.  mask:
    int32 words [B][N][ceil(N / 32)] or [N][...] (tree_mask), None: a chain.
    seg_len: one int32 [B] tensor (or None) per segment of the view: the tokens
    each sequence holds of it."""
    where = "tq_tree_attention"
    _require(q.dim() == 4 and k.dim() == 4 and k.shape == v.shape, where)
    B, N, Hq, d = q.shape
    H = k.shape[1]
    a, b, c = q.stride(), k.stride(), v.stride()
    _require(k.shape == (B, H, N, d) and q.dtype == _F16 and k.dtype == _F16 and v.dtype == _F16 and out.dtype == _F16 and
             out.shape == q.shape and out.is_contiguous() and workspace.is_contiguous() and
             a[3] == b[3] == c[3] == 1, where)
    tensors = [q, k, v, out, workspace]
    mask_ptr, mask_stride = 0, 0
    if mask is not None:
        W = -(-N // 32)
        _require(mask.dtype == _I32 and mask.is_contiguous() and mask.shape in ((N, W), (B, N, W)), where)
        mask_ptr, mask_stride = mask.data_ptr(), N * W if mask.dim() == 3 else 0
        tensors.append(mask)
    lens = [0] * TQ_MAX_SEGMENTS
    if seg_len is not None:
        _require(len(seg_len) == view.n_segments, where)
        for i, n in enumerate(seg_len):
            if n is not None:
                _int32(n, where, (B,))
                lens[i] = n.data_ptr()
                tensors.append(n)
    tree = _pack_tree(N, q.data_ptr(), k.data_ptr(), v.data_ptr(), a[0], a[1], a[2], b[0], b[1], b[2], c[0], c[1], c[2],
                      mask_ptr, mask_stride, *lens, out.data_ptr())
    _call(tensors, stream, where, _lib.tq_tree_attention, ctypes.byref(view), B, H, Hq, d, tree, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out


# ----------------------------------------------------------------- pages
_pack2 = struct.Struct("2q").pack
_pack_pages = [struct.Struct("PqixxxxP" * n).pack for n in range(TQ_MAX_SEGMENTS + 1)]
_pack_verification = struct.Struct("4iPqPqP2qP2qPqPPP").pack
assert struct.calcsize("PqixxxxP") == ctypes.sizeof(tq_pages)
assert struct.calcsize("4iPqPqP2qP2qPqPPP") == ctypes.sizeof(tq_verification)


def _page_args(table, length, count, free_pages, n_free, where):
    B = length.shape[0]
    _require(table.dim() == 2 and length.dim() == 1 and free_pages.dim() == 1, where)
    _int32(table, where, (B, table.shape[1]))
    _int32(length, where, (B,))
    _int32(count, where, (B,))
    _int32(free_pages, where, (free_pages.shape[0],))
    _int32(n_free, where, (1,))
    return B, table.shape[1], table.stride(0) if B > 1 else table.shape[1]


def tq_page_tables(table: torch.Tensor, length: torch.Tensor, n_new: torch.Tensor, free_pages: torch.Tensor,
                   n_free: torch.Tensor, page_size: int, n_max: int, out=None, stream=None):
    """Places for min(n_new[b], n_max) new tokens of each sequence: pages from the stack
    free_pages[:n_free] (int32 [n_pages], [1]) into `table` (int32 [B][max_pages]), length (int32
    [B]) advanced by what was granted.  Returns (slots, positions [B][n_max], granted [B]), int32, -1 behind the
    granted rows; `out`: these three, the first two may be None (not wanted)."""
    where = "tq_page_tables"
    B, width, stride = _page_args(table, length, n_new, free_pages, n_free, where)
    if out is None:
        _require(n_max >= 0 and table.is_cuda, where)
        with on_stream(stream, table.device):
            new = lambda *shape: torch.empty(shape, dtype=_I32, device=table.device)  # noqa: E731
            out = (new(B, n_max), new(B, n_max), new(B))
    slots, positions, granted = out
    _int32(granted, where, (B,))
    for t in (slots, positions):
        _require(t is None or (t.dtype == _I32 and t.shape == (B, n_max) and t.is_contiguous()), where)
    _call([table, length, n_new, free_pages, n_free, granted, slots, positions], stream, where, _lib.tq_page_tables, B,
          page_size, width, free_pages.shape[0], table.data_ptr(), stride, length.data_ptr(), n_new.data_ptr(), n_max,
          free_pages.data_ptr(), n_free.data_ptr(), _ptr(slots), _ptr(positions), granted.data_ptr())
    return out


def tq_page_release(table: torch.Tensor, length: torch.Tensor, keep: torch.Tensor, free_pages: torch.Tensor,
                    n_free: torch.Tensor, page_size: int, stream=None):
    """Sequences cut to min(length[b], keep[b]) tokens (int32 [B]; 0: ended): the pages behind go back onto the
    stack.  Tensors as tq_page_tables takes them."""
    where = "tq_page_release"
    B, width, stride = _page_args(table, length, keep, free_pages, n_free, where)
    _call([table, length, keep, free_pages, n_free], stream, where, _lib.tq_page_release, B, page_size, width,
          free_pages.shape[0], table.data_ptr(), stride, length.data_ptr(), keep.data_ptr(), free_pages.data_ptr(),
          n_free.data_ptr())


def tq_paged_append(pool, rot: tq_rotation | None, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, n_new=None,
                    index=None, n_max: int | None = None, rope: Rope | None = None, positions=None, stream=None):
    """Write rows of K, V (fp16 CUDA [B][H][S][d], unit stride in d) into the pages of `pool` (PackedSegment
    or Fp16Segment of n_pages x page size): row j < min(n_new[b], n_max) of sequence b is source row
    index[b][j] (None: j) and goes to slot slots[b][j] (int32 [B][>= n_max]; outside the pool: skipped).  n_max: default
    the index's width, else the slots' width.  rope, positions, and all else, as tq_append."""
    where = "tq_paged_append"
    L = pool.layout
    shape = K.shape
    _require(len(shape) == 4 and shape == V.shape and K.dtype == _F16 and V.dtype == _F16 and shape[1] == L.n_heads and
             shape[3] == L.head_dim, where)
    a, b = K.stride(), V.stride()
    B, S = shape[0], shape[2]
    _require(a[3] == 1 and b[3] == 1 and slots.dim() == 2, where)
    if n_max is None:
        n_max = index.shape[1] if index is not None else slots.shape[1]
    _int32(slots, where, (B, slots.shape[1]))
    _require(slots.shape[1] >= n_max, where)
    tensors = [K, V, slots, pool.kcodes if pool.kind == TQ_SEG_PACKED else pool.k]
    n_ptr = index_ptr = pos_ptr = rope_ref = None
    index_stride = ps = 0
    if n_new is not None:
        _int32(n_new, where, (B,))
        n_ptr = n_new.data_ptr()
        tensors.append(n_new)
    if index is not None:
        _require(index.dim() == 2 and index.shape[1] >= n_max, where)
        _int32(index, where, (B, index.shape[1]))
        index_ptr, index_stride = index.data_ptr(), index.stride(0)
        tensors.append(index)
    if rope is not None:
        _require(positions is not None, where)
        _int32(positions, where, (S,) if positions.dim() == 1 else (B, S))
        ps = positions.stride(0) if positions.dim() == 2 else 0
        pos_ptr, rope_ref = positions.data_ptr(), rope.ref
        tensors += (positions, rope.table)
    _call(tensors, stream, where, _lib.tq_paged_append, pool.reference(), ctypes.byref(rot) if rot is not None else None,
          rope_ref, pos_ptr, ps, K.data_ptr(), _pack3(a[0], a[1], a[2]), V.data_ptr(), _pack3(b[0], b[1], b[2]), B, S, n_max,
          slots.data_ptr(), slots.stride(0), n_ptr, index_ptr, index_stride)


def tq_paged_read(pool, rot: tq_rotation | None, slots: torch.Tensor, n_read=None, out=None, dtype=torch.float16,
                  stream=None):
    """Rows of the pages of `pool` back as vectors: row j < min(n_read[b], n) of sequence b is slot slots[b][j] (int32
    [B][n]; outside the pool: left as it is).  out, dtype and rot as tq_read takes them ([B][H][n][d])."""
    where = "tq_paged_read"
    L = pool.layout
    _require(slots.dim() == 2, where)
    B, n = slots.shape
    _int32(slots, where, (B, n))
    shape = (B, L.n_heads, n, L.head_dim)
    own = pool.kcodes if pool.kind == TQ_SEG_PACKED else pool.k
    if out is None:
        _require(own.is_cuda, where)
        with on_stream(stream, own.device):  # behind this the kernel writes them
            out = [torch.zeros(shape, dtype=dtype, device=own.device) for _ in range(2)]
    k, v = out
    some = [t for t in (k, v) if t is not None]
    tensors = [slots, own, *some]
    n_ptr = None
    if n_read is not None:
        _int32(n_read, where, (B,))
        n_ptr = n_read.data_ptr()
        tensors.append(n_read)
    if not some:
        return out
    dt = some[0].dtype
    _require(dt in _DTYPE, where)
    args = []
    for t in (k, v):
        if t is None:
            args += (None, None)
            continue
        a = t.stride()
        _require(t.shape == shape and t.dtype == dt and a[3] == 1, where)
        args += (t.data_ptr(), _pack3(a[0], a[1], a[2]))
    _call(tensors, stream, where, _lib.tq_paged_read, pool.reference(), ctypes.byref(rot) if rot is not None else None, B, n,
          slots.data_ptr(), slots.stride(0), n_ptr, _DTYPE[dt], *args)
    return out


def tq_paged_workspace_size(view: tq_layer_view, batch: int, n_heads: int, q_heads: int, head_dim: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.tq_paged_workspace_size(ctypes.byref(view), batch, n_heads, q_heads, head_dim, ctypes.byref(n)),
           "tq_paged_workspace_size")
    return n.value


def tq_paged_attention(view: tq_layer_view, q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, tables, lens,
                       stream=None):
    """out[b][j] = attention of one new token, query head j, over the tokens that sequence b holds of the segments of
    `view`.  q fp16 [B][Hq][d] (unit stride in d), out fp16 [B][Hq][d] contiguous.  tables: per segment int32
    [B][max_pages] (the segment is a pool of pages) or None (it holds sequence b in its batch element b); lens: per
    segment int32 [B] (None: all n_tokens of a segment without a table)."""
    where = "tq_paged_attention"
    _require(q.dim() == 3, where)
    B, Hq, d = q.shape
    n = view.n_segments
    _require(q.dtype == _F16 and out.dtype == _F16 and out.shape == q.shape and out.is_contiguous() and
             workspace.is_contiguous() and (d == 1 or q.stride(2) == 1) and len(tables) == n and len(lens) == n, where)
    tensors = [q, out, workspace]
    fields = []
    for t, c in zip(tables, lens):
        at = stride = width = 0
        if t is not None:
            _require(t.dim() == 2 and c is not None, where)
            width = t.shape[1]
            _int32(t, where, (B, width))
            # (no entries, no storage: a table all the same)
            at, stride = t.data_ptr() if width else c.data_ptr(), t.stride(0) if B > 1 and width else width
            tensors.append(t)
        if c is not None:
            _int32(c, where, (B,))
            tensors.append(c)
        fields += (at, stride, width, 0 if c is None else c.data_ptr())
    H = view.seg[0].layout.n_heads if n else 1  # (no segment: whatever divides the query heads)
    _call(tensors, stream, where, _lib.tq_paged_attention, ctypes.byref(view), _pack_pages[n](*fields), B, H, Hq, d,
          q.data_ptr(), _pack2(q.stride(0), q.stride(1)), out.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out


# ----------------------------------------------------------------- verification of drafts
def tq_verify(tokens: torch.Tensor, target: torch.Tensor, uniform: torch.Tensor, draft: torch.Tensor | None = None,
              parents: torch.Tensor | None = None, out=None, stream=None):
    """Verify drafted tokens (int32 [B][N]; outside the vocabulary: no candidate) against the target's
    probabilities (fp16, bf16 or fp32 [B][N + 1][V]: row 0 behind the last cached token, row i + 1 behind draft i) from
    given random numbers (float32 [B][N + 1], the last for the final token).  draft: the distributions that the drafts were
    drawn from ([B][>= N][V], row 0 the root's children, row i + 1 those of draft i), None: drafts that stand for
    themselves.  parents: int32 [B][N] or [N] (tree_mask takes the same), None: a chain.  Returns (accepted [B][N], n_accepted
    [B], token [B]), int32: the path of accepted drafts (-1 behind it) and the token that follows it."""
    where = "tq_verify"
    _require(tokens.dim() == 2 and target.dim() == 3 and uniform.dim() == 2, where)
    B, N = tokens.shape
    V = target.shape[2]
    _int32(tokens, where, (B, N))
    _require(target.dtype in _DTYPE and target.shape == (B, N + 1, V) and (V == 1 or target.stride(2) == 1), where)
    _require(uniform.dtype == torch.float32 and uniform.shape == (B, N + 1) and (N == 0 or uniform.stride(1) == 1), where)
    tensors = [target, tokens, uniform]
    q_ptr = par_ptr = par_stride = 0
    q_stride = (0, 0)
    if draft is not None:
        _require(draft.dtype == target.dtype and draft.dim() == 3 and draft.shape[0] == B and draft.shape[1] >= N and
                 draft.shape[2] == V and (V == 1 or draft.stride(2) == 1), where)
        q_ptr, q_stride = draft.data_ptr(), draft.stride()[:2]
        tensors.append(draft)
    if parents is not None:
        _int32(parents, where, (N,) if parents.dim() == 1 else (B, N))
        par_ptr, par_stride = parents.data_ptr(), parents.stride(0) if parents.dim() == 2 else 0
        tensors.append(parents)
    if out is None:
        _require(target.is_cuda, where)
        with on_stream(stream, target.device):
            out = tuple(torch.empty(s, dtype=_I32, device=target.device) for s in ((B, N), (B,), (B,)))
    for t, s in zip(out, ((B, N), (B,), (B,))):
        _require(t.dtype == _I32 and t.shape == s and t.is_contiguous(), where)
        tensors.append(t)
    accepted, count, token = out
    _call(tensors, stream, where, _lib.tq_verify,
          _pack_verification(B, N, V, _DTYPE[target.dtype], tokens.data_ptr(), tokens.stride(0), par_ptr, par_stride,
                             target.data_ptr(), target.stride(0), target.stride(1), q_ptr, q_stride[0], q_stride[1],
                             uniform.data_ptr(), uniform.stride(0), accepted.data_ptr(), count.data_ptr(), token.data_ptr()))
    return out
