"""Thin ctypes binding of the C ABI in ``include/pa.h``.

Argument marshalling only: every step of the computation runs in the CUDA
library.  Tensors are torch tensors on the current CUDA device; their data
pointers and element strides are passed through unchanged.  If the library
has not been built, loading raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_SCRATCH_TOO_SMALL = 3
PA_ERR_CUDA = 4
PA_ERR_DEVICE = 5

# bits of the device error code pa_check reports (pa_device_code)
DEVICE_WAIT_TIMEOUT = 1
DEVICE_WORK_OVERFLOW = 2
DEVICE_CAPACITY = 4
DEVICE_PAGE_ID = 8
DEVICE_POSITION = 16

# bytes of the scratch header (error word, then split-arrival counters) at
# the start of every scratch workspace
SCRATCH_HEADER_BYTES = 65536
# (request, kv head group) pairs a plan may have for its last split to merge
MERGE_COUNTERS = (SCRATCH_HEADER_BYTES - 256) // 4

MODE_DECODE = 0
MODE_EXTEND = 1
MODE_VERIFY = 2
KV_BF16 = 0
KV_FP8_E4M3 = 1

EXPORTED_SYMBOLS = ("pa_plan", "pa_decode", "pa_extend", "pa_scratch_init", "pa_check",
                    "pa_status_string", "pa_version", "pa_decode_static_scratch", "pa_append_kv",
                    "pa_debug_wait_expiry", "pa_append_rope_kv", "pa_page_bounds", "pa_sparse_plan",
                    "pa_select_pages", "pa_sparse_attend")


class PaShape(ctypes.Structure):
    _fields_ = [
        ("mode", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("max_batch", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("max_total_q", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("has_sinks", ctypes.c_int32),
        ("soft_cap", ctypes.c_float),
        ("num_splits", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
    ]


class PaPlan(ctypes.Structure):
    _fields_ = [
        ("shape", PaShape),
        ("tile_tokens", ctypes.c_int32),
        ("split_tiles", ctypes.c_int32),
        ("max_splits", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("warps", ctypes.c_int32),
        ("bt_cache", ctypes.c_int32),
        ("smem_bytes", ctypes.c_int32),
        ("grid", ctypes.c_int32 * 3),
        ("scratch_bytes", ctypes.c_int64),
        ("launches", ctypes.c_int32),
        ("kv_copy", ctypes.c_int32),
        ("split_merge", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 5),
    ]


class PaRope(ctypes.Structure):
    _fields_ = [
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("num_axes", ctypes.c_int32),
        ("sections", ctypes.c_int32 * 4),
        ("max_position", ctypes.c_int32),
        ("cos_sin", ctypes.c_void_p),
        ("cos_sin_stride", ctypes.c_int64),
        ("q_norm", ctypes.c_void_p),
        ("k_norm", ctypes.c_void_p),
        ("norm_eps", ctypes.c_float),
        ("norm_offset", ctypes.c_float),
    ]


class PaSparseShape(ctypes.Structure):
    _fields_ = [
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("max_batch", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("max_total_q", ctypes.c_int32),
        ("top_pages", ctypes.c_int32),
        ("first_pages", ctypes.c_int32),
        ("last_pages", ctypes.c_int32),
        ("has_sinks", ctypes.c_int32),
        ("soft_cap", ctypes.c_float),
        ("num_splits", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
    ]


class PaSparsePlan(ctypes.Structure):
    _fields_ = [
        ("shape", PaSparseShape),
        ("tile_tokens", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("warps", ctypes.c_int32),
        ("smem_bytes", ctypes.c_int32),
        ("partial_rows", ctypes.c_int32),
        ("score_rows", ctypes.c_int32),
        ("scratch_bytes", ctypes.c_int64),
        ("reserved", ctypes.c_int32 * 6),
    ]


class PaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the CUDA library (build it first with ``paged_kv_gqa_12_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing "
                           "(run paged_kv_gqa_12_gb300.build.build())")
    L = ctypes.CDLL(path)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    L.pa_plan.argtypes = [ctypes.POINTER(PaShape), vp, i32, ctypes.POINTER(PaPlan)]
    L.pa_plan.restype = ctypes.c_int
    L.pa_decode.argtypes = [ctypes.POINTER(PaPlan), vp, i64, i64, vp, vp, i64, i64, i64, i32, vp, i64,
                            vp, i32, f32, vp, f32, f32, vp, vp, vp, i64, i64, vp, vp, i64, vp]
    L.pa_decode.restype = ctypes.c_int
    L.pa_extend.argtypes = [ctypes.POINTER(PaPlan), vp, i64, i64, vp, vp, i64, i64, i64, i32, vp, i64,
                            vp, vp, i32, i32, f32, vp, f32, f32, vp, vp, vp, i64, i64, vp, vp, i64, vp]
    L.pa_extend.restype = ctypes.c_int
    L.pa_decode_static_scratch.argtypes = [ctypes.POINTER(PaPlan), vp, i64, i64, vp, vp, i64, i64, i64, i32,
                                           vp, i64, vp, i32, f32, vp, f32, f32, vp, i64, i64, vp, vp]
    L.pa_decode_static_scratch.restype = ctypes.c_int
    L.pa_append_kv.argtypes = [vp, vp, i64, i64, vp, vp, i64, i64, i64, i32, i32, i32, i32, i32, vp, i32, f32, f32,
                               vp, vp]
    L.pa_append_kv.restype = ctypes.c_int
    L.pa_append_rope_kv.argtypes = [ctypes.POINTER(PaRope), vp, i64, i64, vp, i64, i64, i32, vp, vp, i64, i64, vp, i64,
                                    vp, vp, i64, i64, i64, i32, i32, i32, i32, i32, vp, i32, f32, f32, vp, vp]
    L.pa_append_rope_kv.restype = ctypes.c_int
    L.pa_page_bounds.argtypes = [vp, i64, i64, i64, i32, i32, i32, i32, i32, vp, i64, i32, vp, vp, i32, f32, vp, vp,
                                 i64, i64, vp, vp]
    L.pa_page_bounds.restype = ctypes.c_int
    L.pa_sparse_plan.argtypes = [ctypes.POINTER(PaSparseShape), ctypes.POINTER(PaSparsePlan)]
    L.pa_sparse_plan.restype = ctypes.c_int
    L.pa_select_pages.argtypes = [ctypes.POINTER(PaSparsePlan), vp, i64, i64, vp, i64, i64, i32, vp, i64, vp, vp, i32,
                                  i32, vp, vp, i64, vp]
    L.pa_select_pages.restype = ctypes.c_int
    L.pa_sparse_attend.argtypes = [ctypes.POINTER(PaSparsePlan), vp, i64, i64, vp, vp, i64, i64, i64, i32, vp, i64,
                                   vp, vp, i32, i32, vp, f32, vp, f32, f32, vp, vp, vp, i64, i64, vp, vp, i64, vp]
    L.pa_sparse_attend.restype = ctypes.c_int
    L.pa_debug_wait_expiry.argtypes = [vp, i32, i64, vp]
    L.pa_debug_wait_expiry.restype = ctypes.c_int
    L.pa_scratch_init.argtypes = [vp, vp]
    L.pa_scratch_init.restype = ctypes.c_int
    L.pa_check.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
    L.pa_check.restype = ctypes.c_int
    L.pa_status_string.argtypes = [ctypes.c_int]
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_version.argtypes = []
    L.pa_version.restype = i32
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, where: str):
    if status != PA_OK:
        raise PaError(status, where)


def plan(*, mode: int, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
         kv_dtype: int = KV_BF16, max_batch: int, max_pages_per_seq: int, max_total_q: int = 0,
         window: int = 0, has_sinks: bool = False, soft_cap: float = 0.0, num_splits: int = 0,
         num_sms: int = 0, q_len: int = 0, host_seq_lens=None) -> PaPlan:
    """pa_plan.  ``host_seq_lens``: optional host int32 sequence of lengths."""
    s = PaShape(mode=mode, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim,
                page_size=page_size, kv_dtype=kv_dtype, max_batch=max_batch,
                max_pages_per_seq=max_pages_per_seq, max_total_q=max_total_q, window=window,
                has_sinks=1 if has_sinks else 0, soft_cap=soft_cap, num_splits=num_splits, num_sms=num_sms,
                q_len=q_len)
    p = PaPlan()
    lens_arr, n = None, 0
    if host_seq_lens is not None:
        vals = [int(x) for x in host_seq_lens]
        n = len(vals)
        lens_arr = (ctypes.c_int32 * max(n, 1))(*vals)
    _check(load().pa_plan(ctypes.byref(s), lens_arr, n, ctypes.byref(p)), "pa_plan")
    return p


def _kv_strides(k_cache, v_cache):
    if tuple(k_cache.stride()) != tuple(v_cache.stride()) or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must share shape and strides")
    if k_cache.dim() != 4 or k_cache.stride(3) != 1:
        raise ValueError("caches must be [pages, page_size, kv_heads, head_dim] with contiguous head_dim")
    return k_cache.stride(0), k_cache.stride(1), k_cache.stride(2)


def decode(p: PaPlan, q, k_cache, v_cache, block_table, seq_lens, *, scale: float, out, lse=None,
           sinks=None, k_scale: float = 1.0, v_scale: float = 1.0, k_scales=None, v_scales=None, scratch,
           stream=None):
    """pa_decode on torch tensors (q/out [B, Hq, D] bf16; caches bf16 or uint8 e4m3;
    k_scales / v_scales: optional device fp32 [B] per-request descales)."""
    sp, st, sh = _kv_strides(k_cache, v_cache)
    status = load().pa_decode(
        ctypes.byref(p), _ptr(q), q.stride(0), q.stride(1), _ptr(k_cache), _ptr(v_cache), sp, st, sh,
        k_cache.shape[0], _ptr(block_table), block_table.stride(0), _ptr(seq_lens), seq_lens.shape[0],
        float(scale), _ptr(sinks), float(k_scale), float(v_scale), _ptr(k_scales), _ptr(v_scales), _ptr(out),
        out.stride(0), out.stride(1), _ptr(lse), _ptr(scratch), scratch.numel() * scratch.element_size(),
        _stream(stream))
    _check(status, "pa_decode")


def extend(p: PaPlan, q, k_cache, v_cache, block_table, seq_lens, query_start_loc, *, scale: float, out,
           lse=None, sinks=None, k_scale: float = 1.0, v_scale: float = 1.0, k_scales=None, v_scales=None,
           scratch, stream=None):
    """pa_extend on torch tensors (q/out [T, Hq, D] bf16; k_scales / v_scales:
    optional device fp32 [B] per-request descales)."""
    sp, st, sh = _kv_strides(k_cache, v_cache)
    status = load().pa_extend(
        ctypes.byref(p), _ptr(q), q.stride(0), q.stride(1), _ptr(k_cache), _ptr(v_cache), sp, st, sh,
        k_cache.shape[0], _ptr(block_table), block_table.stride(0), _ptr(seq_lens), _ptr(query_start_loc),
        seq_lens.shape[0], q.shape[0], float(scale), _ptr(sinks), float(k_scale), float(v_scale), _ptr(k_scales),
        _ptr(v_scales), _ptr(out), out.stride(0), out.stride(1), _ptr(lse), _ptr(scratch),
        scratch.numel() * scratch.element_size(), _stream(stream))
    _check(status, "pa_extend")


def decode_static_scratch(p: PaPlan, q, k_cache, v_cache, block_table, seq_lens, *, scale: float, out,
                          lse=None, sinks=None, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """pa_decode_static_scratch: decode for callers that cannot allocate a
    workspace; the library's own fixed 16 MiB device array is used instead
    (calls on one device must not overlap)."""
    sp, st, sh = _kv_strides(k_cache, v_cache)
    status = load().pa_decode_static_scratch(
        ctypes.byref(p), _ptr(q), q.stride(0), q.stride(1), _ptr(k_cache), _ptr(v_cache), sp, st, sh,
        k_cache.shape[0], _ptr(block_table), block_table.stride(0), _ptr(seq_lens), seq_lens.shape[0],
        float(scale), _ptr(sinks), float(k_scale), float(v_scale), _ptr(out), out.stride(0), out.stride(1),
        _ptr(lse), _stream(stream))
    _check(status, "pa_decode_static_scratch")


def append_kv(k_new, v_new, k_cache, v_cache, slot_mapping, *, kv_dtype: int = KV_BF16, k_scale: float = 1.0,
              v_scale: float = 1.0, scratch=None, stream=None):
    """pa_append_kv: write new tokens' K/V (bf16 [T, Hkv, D]) into the paged caches at slot_mapping (int64)."""
    sp, st, sh = _kv_strides(k_cache, v_cache)
    if tuple(k_new.stride()) != tuple(v_new.stride()) or k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must share shape and strides")
    status = load().pa_append_kv(
        _ptr(k_new), _ptr(v_new), k_new.stride(0), k_new.stride(1), _ptr(k_cache), _ptr(v_cache), sp, st, sh,
        k_cache.shape[0], k_cache.shape[1], k_cache.shape[2], k_cache.shape[3], int(kv_dtype), _ptr(slot_mapping),
        k_new.shape[0], float(k_scale), float(v_scale), _ptr(scratch), _stream(stream))
    _check(status, "pa_append_kv")


def rope(cos_sin=None, *, rot_dim: int, interleaved: bool = False, sections=None, q_norm=None, k_norm=None,
         norm_eps: float = 1e-6, norm_offset: float = 0.0) -> PaRope:
    """Norm and rotation for append_rope_kv.  ``cos_sin``: fp32 [max_position, rot_dim] (cosines, then sines; None
    with rot_dim 0); ``sections``: pairs per position axis (None: one axis); ``q_norm`` / ``k_norm``: bf16 [head_dim]
    RMS norm weights or None.  The tensors are kept alive by the returned struct."""
    if (cos_sin is None) != (rot_dim == 0):
        raise ValueError("cos_sin is given exactly when rot_dim > 0")
    sec = [int(x) for x in sections] if sections is not None else [rot_dim // 2]
    if not 1 <= len(sec) <= 4:
        raise ValueError("1 to 4 position axes")
    if min(sec) < 0 or sum(sec) != rot_dim // 2:
        raise ValueError("sections must sum to rot_dim / 2")
    dev = _device(*(t for t in (cos_sin, q_norm, k_norm) if t is not None))
    for name, t, dtype, dims in (("q_norm", q_norm, torch.bfloat16, 1), ("k_norm", k_norm, torch.bfloat16, 1),
                                 ("cos_sin", cos_sin, torch.float32, 2)):
        if t is not None:
            _typed(name, t, dtype, dims, dev)
    if cos_sin is not None and cos_sin.shape[1] != rot_dim:
        raise ValueError("cos_sin must be [max_position, rot_dim]")
    r = PaRope(rot_dim=rot_dim, interleaved=1 if interleaved else 0, num_axes=len(sec),
               sections=(ctypes.c_int32 * 4)(*sec), max_position=0 if cos_sin is None else cos_sin.shape[0],
               cos_sin=_ptr(cos_sin), cos_sin_stride=0 if cos_sin is None else cos_sin.stride(0), q_norm=_ptr(q_norm),
               k_norm=_ptr(k_norm), norm_eps=float(norm_eps), norm_offset=float(norm_offset))
    dims = {t.shape[0] for t in (q_norm, k_norm) if t is not None}
    if len(dims) > 1:
        raise ValueError("q_norm and k_norm must be [head_dim]")
    r.tensors = (cos_sin, q_norm, k_norm)
    if dev >= 0:
        r.device = dev
    if dims:
        r.norm_dim = dims.pop()
    return r


# A call of a few microseconds on the GPU should not wait for its checks: each
# function compares a tensor's type, device and strides in place and leaves what
# does not look as usual to _typed, which decides and words the error.

_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _device(*tensors) -> int:
    """The current CUDA device, which the first tensor (or none) has to be on."""
    if tensors and tensors[0].get_device() < 0:
        raise ValueError("tensors must be on the current CUDA device")
    return torch._C._cuda_getDevice() if tensors else -1


def _typed(name, t, dtype, dims, dev):
    """Refuse a tensor of another type, rank or device, or without a contiguous innermost dimension."""
    if t.dtype is not dtype or t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-d {dtype} tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    if t.stride(dims - 1) != 1 and t.shape[dims - 1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _raw_stream(stream, dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _pair(k_name, k, v_name, v, dtype, dims, dev):
    """Two tensors of one type, shape and strides; returns both tuples."""
    shape, stride = k.shape, k.stride()
    if k.dtype is not dtype or v.dtype is not dtype or k.get_device() != dev or v.get_device() != dev \
            or len(stride) != dims or stride[-1] != 1:
        _typed(k_name, k, dtype, dims, dev)
        _typed(v_name, v, dtype, dims, dev)
    if v.stride() != stride or v.shape != shape:
        raise ValueError(f"{k_name} and {v_name} must share shape and strides")
    return shape, stride


def _scratch(scratch, dev):
    """Pointer of a workspace (alloc_scratch makes one); the call itself checks its size."""
    if scratch.get_device() != dev or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous tensor on the current CUDA device")
    return scratch.data_ptr()


def _header(scratch, dev):
    """Pointer of an optional workspace of which the header alone is used."""
    if scratch is None:
        return None
    if scratch.nbytes < SCRATCH_HEADER_BYTES:
        raise ValueError(f"scratch must hold the header's {SCRATCH_HEADER_BYTES} bytes")
    return _scratch(scratch, dev)


def _cache_type(kv_dtype):
    return torch.uint8 if kv_dtype == KV_FP8_E4M3 else _BF16


def append_rope_kv(r: PaRope, k_new, v_new, positions, k_cache, v_cache, slot_mapping, *, q=None, q_out=None,
                   kv_dtype: int = KV_BF16, k_scale: float = 1.0, v_scale: float = 1.0, scratch=None, stream=None):
    """pa_append_rope_kv: norm and rotate q (bf16 [T, Hq, D], into q_out) and k_new (bf16 [T, Hkv, D]), write k_new
    and v_new into the paged caches at slot_mapping (int64 [T]).  positions: int32 [T], or [axes, T]."""
    dev = _device(k_new)
    (T, hkv, D), ns = _pair("k_new", k_new, "v_new", v_new, _BF16, 3, dev)
    cs, kvs = _pair("k_cache", k_cache, "v_cache", v_cache, _cache_type(kv_dtype), 4, dev)
    if slot_mapping.dtype is not _I64 or slot_mapping.get_device() != dev or slot_mapping.stride() != (1,):
        _typed("slot_mapping", slot_mapping, _I64, 1, dev)
    if cs[2] != hkv or cs[3] != D or slot_mapping.shape[0] != T:
        raise ValueError("k_new must be [tokens, kv_heads, head_dim] of the cache, slot_mapping [tokens]")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    hq, qp, qs, op, os_ = 0, None, (0, 0), None, (0, 0)
    if q is not None:
        shape, qs, os_ = q.shape, q.stride(), q_out.stride()
        if q.dtype is not _BF16 or q_out.dtype is not _BF16 or q.get_device() != dev or q_out.get_device() != dev \
                or len(qs) != 3 or qs[-1] != 1 or len(os_) != 3 or os_[-1] != 1:
            _typed("q", q, _BF16, 3, dev)
            _typed("q_out", q_out, _BF16, 3, dev)
        if q_out.shape != shape or shape[0] != T or shape[2] != D:
            raise ValueError("q and q_out must be [tokens, q_heads, head_dim]")
        hq, qp, op = shape[1], q.data_ptr(), q_out.data_ptr()
    if getattr(r, "norm_dim", D) != D:
        raise ValueError("q_norm and k_norm must be [head_dim]")
    if getattr(r, "device", dev) != dev:
        raise ValueError("cos_sin, q_norm and k_norm must be on the current CUDA device")
    pp, ps = None, 0
    if r.rot_dim > 0:
        if positions is None:
            raise ValueError("a rotation needs positions")
        shape, stride, axes = positions.shape, positions.stride(), r.num_axes
        if positions.dtype is not _I32 or positions.get_device() != dev or stride[-1] != 1:
            _typed("positions", positions, _I32, len(shape), dev)
        if shape != (axes, T) and not (axes == 1 and shape == (T,)):
            raise ValueError("positions must be [axes, tokens] ([tokens] for one axis)")
        pp, ps = positions.data_ptr(), stride[0] if len(stride) == 2 else T
    status = load().pa_append_rope_kv(
        ctypes.byref(r), qp, qs[0], qs[1], op, os_[0], os_[1], hq, k_new.data_ptr(), v_new.data_ptr(), ns[0], ns[1], pp,
        ps, k_cache.data_ptr(), v_cache.data_ptr(), kvs[0], kvs[1], kvs[2], cs[0], cs[1], hkv, D, kv_dtype,
        slot_mapping.data_ptr(), T, k_scale, v_scale, _header(scratch, dev),
        _raw_stream(stream, dev))
    if status != PA_OK:
        raise PaError(status, "pa_append_rope_kv")


def _requests(block_table, seq_lens, query_start_loc, dev):
    """Checks of the request metadata; returns (batch, block-table row stride and width)."""
    batch, bts, (rows, width) = seq_lens.shape[0], block_table.stride(), block_table.shape
    if block_table.dtype is not _I32 or block_table.get_device() != dev or bts[-1] != 1:
        _typed("block_table", block_table, _I32, 2, dev)
    if seq_lens.dtype is not _I32 or seq_lens.get_device() != dev or seq_lens.stride() != (1,):
        _typed("seq_lens", seq_lens, _I32, 1, dev)
    if rows < batch:
        raise ValueError("block_table must have a row per request")
    if query_start_loc is not None:
        if query_start_loc.dtype is not _I32 or query_start_loc.get_device() != dev or query_start_loc.stride() != (1,):
            _typed("query_start_loc", query_start_loc, _I32, 1, dev)
        if query_start_loc.shape[0] != batch + 1:
            raise ValueError("query_start_loc must be [batch + 1]")
    return batch, bts[0], width


def _bounds(bounds, pages, kv_heads, head_dim, dev):
    """Checks of a bounds tensor; returns its strides."""
    s = bounds.stride()
    if bounds.dtype is not _BF16 or bounds.get_device() != dev or len(s) != 4 or s[-1] != 1:
        _typed("bounds", bounds, _BF16, 4, dev)
    if bounds.shape != (pages, kv_heads, 2, head_dim) or s[2] != head_dim:
        raise ValueError("bounds must be [pages, kv_heads, 2, head_dim], the last two dimensions contiguous")
    return s


def _floats(name, t, n, dev):
    """Pointer of an optional fp32 [n] tensor."""
    if t is None:
        return None
    _typed(name, t, _F32, 1, dev)
    if t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}]")
    return t.data_ptr()


def page_bounds(k_cache, block_table, seq_lens, bounds, *, query_start_loc=None, kv_dtype: int = KV_BF16,
                k_scale: float = 1.0, k_scales=None, scratch=None, stream=None):
    """pa_page_bounds: refresh bounds (bf16 [pages, kv_heads, 2, head_dim]: smallest, largest key value per dim) of
    the pages that hold new tokens (query_start_loc), or of every page of the requests (None)."""
    dev = _device(k_cache)
    ks, dtype = k_cache.stride(), _cache_type(kv_dtype)
    if k_cache.dtype is not dtype or k_cache.get_device() != dev or len(ks) != 4 or ks[-1] != 1:
        _typed("k_cache", k_cache, dtype, 4, dev)
    batch, bts, width = _requests(block_table, seq_lens, query_start_loc, dev)
    pages, ps, hkv, D = k_cache.shape
    bs = _bounds(bounds, pages, hkv, D, dev)
    status = load().pa_page_bounds(
        k_cache.data_ptr(), ks[0], ks[1], ks[2], pages, ps, hkv, D, kv_dtype, block_table.data_ptr(), bts, width,
        seq_lens.data_ptr(), None if query_start_loc is None else query_start_loc.data_ptr(), batch, k_scale,
        _floats("k_scales", k_scales, batch, dev), bounds.data_ptr(), bs[0], bs[1],
        _header(scratch, dev), _raw_stream(stream, dev))
    if status != PA_OK:
        raise PaError(status, "pa_page_bounds")


def sparse_plan(*, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, kv_dtype: int = KV_BF16,
                max_batch: int, max_pages_per_seq: int, max_total_q: int, top_pages: int, first_pages: int = 1,
                last_pages: int = 2, has_sinks: bool = False, soft_cap: float = 0.0, num_splits: int = 0,
                num_sms: int = 0) -> PaSparsePlan:
    """pa_sparse_plan: the plan of select_pages and sparse_attend."""
    s = PaSparseShape(num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim, page_size=page_size,
                      kv_dtype=kv_dtype, max_batch=max_batch, max_pages_per_seq=max_pages_per_seq,
                      max_total_q=max_total_q, top_pages=top_pages, first_pages=first_pages, last_pages=last_pages,
                      has_sinks=1 if has_sinks else 0, soft_cap=soft_cap, num_splits=num_splits, num_sms=num_sms)
    p = PaSparsePlan()
    _check(load().pa_sparse_plan(ctypes.byref(s), ctypes.byref(p)), "pa_sparse_plan")
    return p


def _sparse_rows(s, q, pages, block_table, seq_lens, query_start_loc, dev):
    """Checks of query rows and their page lists against a plan's shape; returns (rows, q strides, batch, block-table
    row stride)."""
    hkv, top, qs = s.num_kv_heads, s.top_pages, q.stride()
    if q.dtype is not _BF16 or q.get_device() != dev or len(qs) != 3 or qs[-1] != 1:
        _typed("q", q, _BF16, 3, dev)
    if pages.dtype is not _I32 or pages.get_device() != dev or len(pages.shape) != 3:
        _typed("pages", pages, _I32, 3, dev)
    batch, bts, width = _requests(block_table, seq_lens, query_start_loc, dev)
    rows, hq, D = q.shape
    if hq != s.num_q_heads or D != s.head_dim:
        raise ValueError("q must be [rows, q_heads, head_dim] of the plan")
    if pages.shape != (rows, hkv, top) or (pages.stride() != (hkv * top, top, 1) and not pages.is_contiguous()):
        raise ValueError("pages must be contiguous [rows, kv_heads, top_pages] of the plan")
    if width < s.max_pages_per_seq:
        raise ValueError("block_table must be max_pages_per_seq of the plan wide")
    return rows, qs, batch, bts


def select_pages(p: PaSparsePlan, q, bounds, block_table, seq_lens, pages, *, query_start_loc=None, scratch,
                 stream=None):
    """pa_select_pages: pages (int32 [rows, kv_heads, top_pages]) of each query row (bf16 q [rows, Hq, D]) by the key
    bounds page_bounds wrote.  One row per request without query_start_loc, packed rows with it."""
    dev, s = _device(q), p.shape
    rows, qs, batch, bts = _sparse_rows(s, q, pages, block_table, seq_lens, query_start_loc, dev)
    pool = bounds.shape[0]
    bs = _bounds(bounds, pool, s.num_kv_heads, s.head_dim, dev)
    status = load().pa_select_pages(
        ctypes.byref(p), q.data_ptr(), qs[0], qs[1], bounds.data_ptr(), bs[0], bs[1], pool, block_table.data_ptr(), bts,
        seq_lens.data_ptr(), None if query_start_loc is None else query_start_loc.data_ptr(), batch, rows,
        pages.data_ptr(), _scratch(scratch, dev), scratch.nbytes, _raw_stream(stream, dev))
    if status != PA_OK:
        raise PaError(status, "pa_select_pages")


def sparse_attend(p: PaSparsePlan, q, k_cache, v_cache, block_table, seq_lens, pages, *, query_start_loc=None,
                  scale: float, out, lse=None, sinks=None, k_scale: float = 1.0, v_scale: float = 1.0, k_scales=None,
                  v_scales=None, scratch, stream=None):
    """pa_sparse_attend: attention of each query row over the pages chosen for it (q / out bf16 [rows, Hq, D], lse
    fp32 [rows, Hq])."""
    dev, s = _device(q), p.shape
    rows, qs, batch, bts = _sparse_rows(s, q, pages, block_table, seq_lens, query_start_loc, dev)
    (pool, ps, hkv, D), kvs = _pair("k_cache", k_cache, "v_cache", v_cache, _cache_type(s.kv_dtype), 4, dev)
    if ps != s.page_size or hkv != s.num_kv_heads or D != s.head_dim:
        raise ValueError("caches must be [pages, page_size, kv_heads, head_dim] of the plan")
    os_ = out.stride()
    if out.dtype is not _BF16 or out.get_device() != dev or len(os_) != 3 or os_[-1] != 1:
        _typed("out", out, _BF16, 3, dev)
    if out.shape != q.shape:
        raise ValueError("out must be [rows, q_heads, head_dim]")
    if lse is not None:
        hq = s.num_q_heads
        if lse.dtype is not _F32 or lse.get_device() != dev or len(lse.shape) != 2:
            _typed("lse", lse, _F32, 2, dev)
        if lse.shape != (rows, hq) or (lse.stride() != (hq, 1) and not lse.is_contiguous()):
            raise ValueError("lse must be contiguous [rows, q_heads]")
    status = load().pa_sparse_attend(
        ctypes.byref(p), q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(), kvs[0], kvs[1], kvs[2],
        pool, block_table.data_ptr(), bts, seq_lens.data_ptr(),
        None if query_start_loc is None else query_start_loc.data_ptr(), batch, rows, pages.data_ptr(), scale,
        _floats("sinks", sinks, s.num_q_heads, dev), k_scale, v_scale, _floats("k_scales", k_scales, batch, dev),
        _floats("v_scales", v_scales, batch, dev), out.data_ptr(), os_[0], os_[1],
        None if lse is None else lse.data_ptr(), _scratch(scratch, dev), scratch.nbytes, _raw_stream(stream, dev))
    if status != PA_OK:
        raise PaError(status, "pa_sparse_attend")


def debug_wait_expiry(scratch, which: int, limit_ns: int, stream=None):
    """pa_debug_wait_expiry: run one bounded device wait out on purpose (test hook)."""
    _check(load().pa_debug_wait_expiry(_ptr(scratch), int(which), int(limit_ns), _stream(stream)),
           "pa_debug_wait_expiry")


def scratch_init(scratch, stream=None):
    _check(load().pa_scratch_init(_ptr(scratch), _stream(stream)), "pa_scratch_init")


def check(scratch, stream=None) -> int:
    """pa_check: synchronises and returns the device error code (0 = none)."""
    code = ctypes.c_uint32(0)
    status = load().pa_check(_ptr(scratch), _stream(stream), ctypes.byref(code))
    if status not in (PA_OK, PA_ERR_DEVICE):
        raise PaError(status, "pa_check")
    return int(code.value)


def alloc_scratch(p: PaPlan, device=None):
    """Allocate a scratch workspace (torch uint8, 256-byte aligned) for a plan
    and zero its error header."""
    n = int(p.scratch_bytes)
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-buf.data_ptr()) % 256
    s = buf[off:off + n]
    scratch_init(s)
    return s
