"""Thin Python binding of libtactkv.so (include/tactkv.h): argument marshalling only.

Every step of compression and decompression runs in the library's CUDA kernels.  PyTorch is
used for device memory and streams: the helpers below allocate payload, output and workspace
tensors and pass their device pointers to the C ABI.  If the shared library is missing the
import fails; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtactkv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m dct_transform_coding_b200.build` "
                      "(or __graft_entry__.build()); the codec has no CPU path")
_lib = ctypes.CDLL(LIB_PATH)

TACTKV_OK = 0
TACTKV_INVALID_ARG = 1
TACTKV_UNSUPPORTED_SHAPE = 2
TACTKV_CAPACITY = 3
TACTKV_ALIGNMENT = 4
TACTKV_CORRUPT_PAYLOAD = 5
TACTKV_CUDA = 6
TACTKV_WORKSPACE = 7
TACTKV_SCRATCH_LIMIT = 8
TACTKV_TIMEOUT = 9

TACTKV_NO_QUANT = 1
TACTKV_FP32_IO = 2
TACTKV_SKIP_S = 4
TACTKV_SKIP_H = 8
TACTKV_SKIP_W = 16
TACTKV_UNIFORM_ALLOC = 32
TACTKV_ROTATE = 64
TACTKV_HEAD_GAIN = 128

TACTKV_TEXT_BF16 = 0
TACTKV_TEXT_MXFP8 = 1
TACTKV_TEXT_MXFP4 = 2
TEXT_FORMATS = {"bf16": TACTKV_TEXT_BF16, "mxfp8": TACTKV_TEXT_MXFP8, "mxfp4": TACTKV_TEXT_MXFP4}

HEADER_BYTES = 64
EXPORTED = ("tactkv_payload_bytes", "tactkv_workspace_bytes", "tactkv_compress", "tactkv_decompress",
            "tactkv_compress_profiled", "tactkv_decompress_profiled", "tactkv_compress_noalloc",
            "tactkv_allocate", "tactkv_device_status", "tactkv_occupancy", "tactkv_max_batch",
            "tactkv_attention_workspace_bytes", "tactkv_attention_decode",
            "tactkv_text_workspace_bytes", "tactkv_text_append", "tactkv_text_read", "tactkv_text_attention",
            "tactkv_status_string", "tactkv_lloyd_max_table", "tactkv_format_version", "tactkv_last_launches")


class tactkv_unit(ctypes.Structure):
    _fields_ = [
        ("layer", ctypes.c_int32), ("kv", ctypes.c_int32),
        ("S", ctypes.c_int32), ("H", ctypes.c_int32), ("W", ctypes.c_int32),
        ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("bits", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("kv_in", ctypes.c_void_p), ("kv_out", ctypes.c_void_p),
        ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
        ("payload", ctypes.c_void_p), ("payload_capacity", ctypes.c_size_t),
    ]


class tactkv_occupancy_t(ctypes.Structure):
    _fields_ = [("bins", ctypes.c_uint64), ("channels", ctypes.c_uint64), ("code_bits", ctypes.c_uint64),
                ("formula_bits", ctypes.c_uint64), ("index_bits", ctypes.c_uint64),
                ("payload_bytes", ctypes.c_uint64), ("bits_per_element", ctypes.c_double),
                ("shrink_vs_bf16", ctypes.c_double)]


class tactkv_text_cache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("k_pages", ctypes.c_void_p),
                ("v_pages", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class tactkv_text_batch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("row_starts", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_P = ctypes.POINTER(tactkv_unit)
_TC, _TB = ctypes.c_void_p, ctypes.c_void_p   # tactkv_text_cache and tactkv_text_batch, as addresses or packed bytes
_lib.tactkv_payload_bytes.restype = ctypes.c_size_t
_lib.tactkv_payload_bytes.argtypes = [_P]
_lib.tactkv_workspace_bytes.restype = ctypes.c_size_t
_lib.tactkv_workspace_bytes.argtypes = [_P, ctypes.c_int]
for _name in ("tactkv_compress", "tactkv_decompress"):
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = [_P, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
for _name in ("tactkv_compress_profiled", "tactkv_decompress_profiled"):
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = [_P, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                     ctypes.POINTER(ctypes.c_void_p)]
_lib.tactkv_compress_noalloc.restype = ctypes.c_int
_lib.tactkv_compress_noalloc.argtypes = [_P, ctypes.c_int, ctypes.c_void_p]
_lib.tactkv_allocate.restype = ctypes.c_int
_lib.tactkv_allocate.argtypes = [_P, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
_lib.tactkv_device_status.restype = ctypes.c_int
_lib.tactkv_device_status.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
_lib.tactkv_occupancy.restype = ctypes.c_int
_lib.tactkv_occupancy.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(tactkv_occupancy_t)]
_lib.tactkv_max_batch.restype = ctypes.c_int64
_lib.tactkv_max_batch.argtypes = [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint64]
_lib.tactkv_attention_workspace_bytes.restype = ctypes.c_size_t
_lib.tactkv_attention_workspace_bytes.argtypes = [_P, ctypes.c_int, ctypes.c_int]
_lib.tactkv_attention_decode.restype = ctypes.c_int
_lib.tactkv_attention_decode.argtypes = [_P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]
_lib.tactkv_text_workspace_bytes.restype = ctypes.c_size_t
_lib.tactkv_text_workspace_bytes.argtypes = [_TC] + [ctypes.c_int] * 5
_lib.tactkv_text_append.restype = ctypes.c_int
_lib.tactkv_text_append.argtypes = [_TC, _TB, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t,
                                    ctypes.c_void_p]
_lib.tactkv_text_read.restype = ctypes.c_int
_lib.tactkv_text_read.argtypes = [_TC, _TB, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                  ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
_lib.tactkv_text_attention.restype = ctypes.c_int
_lib.tactkv_text_attention.argtypes = [_TC, _TB, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int64] + [ctypes.c_void_p] * 7 + [
                                       ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
_lib.tactkv_status_string.restype = ctypes.c_char_p
_lib.tactkv_status_string.argtypes = [ctypes.c_int]
_lib.tactkv_lloyd_max_table.restype = ctypes.c_int
_lib.tactkv_lloyd_max_table.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]
_lib.tactkv_format_version.restype = ctypes.c_int
_lib.tactkv_format_version.argtypes = []
_lib.tactkv_last_launches.restype = ctypes.c_int
_lib.tactkv_last_launches.argtypes = []


class TactkvError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {tactkv_status_string(status)} ({status})")


# ------------------------------------------------------------------------- raw C entry points ---
def tactkv_payload_bytes(unit: tactkv_unit) -> int:
    return int(_lib.tactkv_payload_bytes(ctypes.byref(unit)))


def tactkv_workspace_bytes(units) -> int:
    arr = _as_array(units)
    return int(_lib.tactkv_workspace_bytes(arr, len(arr)))


def tactkv_compress(units, workspace_ptr: int, workspace_bytes: int, stream_ptr: int) -> int:
    arr = _as_array(units)
    return int(_lib.tactkv_compress(arr, len(arr), ctypes.c_void_p(workspace_ptr), workspace_bytes,
                                    ctypes.c_void_p(stream_ptr)))


def tactkv_decompress(units, workspace_ptr: int, workspace_bytes: int, stream_ptr: int) -> int:
    arr = _as_array(units)
    return int(_lib.tactkv_decompress(arr, len(arr), ctypes.c_void_p(workspace_ptr), workspace_bytes,
                                      ctypes.c_void_p(stream_ptr)))


def _events_array(events):
    if events is None:
        return None
    return (ctypes.c_void_p * len(events))(*[int(e) if e else None for e in events])


def tactkv_compress_profiled(units, workspace_ptr: int, workspace_bytes: int, stream_ptr: int, events) -> int:
    """events: sequence of 5 cudaEvent_t handles (ints, e.g. torch.cuda.Event().cuda_event) or None."""
    arr = _as_array(units)
    return int(_lib.tactkv_compress_profiled(arr, len(arr), ctypes.c_void_p(workspace_ptr), workspace_bytes,
                                             ctypes.c_void_p(stream_ptr), _events_array(events)))


def tactkv_decompress_profiled(units, workspace_ptr: int, workspace_bytes: int, stream_ptr: int, events) -> int:
    """events: sequence of 4 cudaEvent_t handles or None."""
    arr = _as_array(units)
    return int(_lib.tactkv_decompress_profiled(arr, len(arr), ctypes.c_void_p(workspace_ptr), workspace_bytes,
                                               ctypes.c_void_p(stream_ptr), _events_array(events)))


def tactkv_compress_noalloc(units, stream_ptr: int) -> int:
    """Compress with the library's fixed device scratch instead of a caller workspace (for callers
    that cannot allocate, e.g. while recording a CUDA graph).  Calls share that scratch: serialize
    calls that could overlap on the GPU."""
    arr = _as_array(units)
    return int(_lib.tactkv_compress_noalloc(arr, len(arr), ctypes.c_void_p(stream_ptr)))


def tactkv_allocate(unit: tactkv_unit, var_ptr: int, workspace_ptr: int, workspace_bytes: int,
                    stream_ptr: int) -> int:
    """Stage 3 on given fp64 variances (device pointer var_ptr, N doubles): header, b[] and sigma[]
    of unit.payload as compress would write them."""
    return int(_lib.tactkv_allocate(ctypes.byref(unit), ctypes.c_void_p(var_ptr), ctypes.c_void_p(workspace_ptr),
                                    workspace_bytes, ctypes.c_void_p(stream_ptr)))


def allocate(var: torch.Tensor, S: int, H: int, W: int, bits: int, *, heads: int = 1, head_dim: int = 32,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Bit allocation of the fp64 variances var [S*H*W] (on the GPU): returns b [S*H*W] uint8."""
    var = var.to(torch.float64).contiguous()
    cap = payload_capacity(S, H, W, heads, head_dim, bits)
    payload = torch.zeros(((cap + 15) // 16 * 16,), dtype=torch.uint8, device=var.device)
    u = tactkv_unit(S=S, H=H, W=W, heads=heads, head_dim=head_dim, bits=bits, payload=payload.data_ptr(),
                    payload_capacity=payload.numel(), token_stride=heads * head_dim, head_stride=head_dim)
    ws = alloc_workspace([u], var.device)
    st = tactkv_allocate(u, var.data_ptr(), ws.data_ptr(), ws.numel(), _stream_ptr(stream))
    if st != TACTKV_OK:
        raise TactkvError(st, "tactkv_allocate")
    N = S * H * W
    return payload[HEADER_BYTES:HEADER_BYTES + N]


def tactkv_attention_workspace_bytes(k_units, n_units: int, q_heads: int) -> int:
    return int(_lib.tactkv_attention_workspace_bytes(_as_array(k_units), n_units, q_heads))


def tactkv_device_status(workspace_ptr: int, workspace_bytes: int, stream_ptr: int) -> int:
    return int(_lib.tactkv_device_status(ctypes.c_void_p(workspace_ptr), workspace_bytes, ctypes.c_void_p(stream_ptr)))


def tactkv_occupancy(payload) -> dict:
    """Occupancy of one payload (a host bytes-like object or a CPU uint8 tensor)."""
    buf = bytes(payload.numpy().tobytes()) if isinstance(payload, torch.Tensor) else bytes(payload)
    out = tactkv_occupancy_t()
    st = int(_lib.tactkv_occupancy(ctypes.c_char_p(buf), len(buf), ctypes.byref(out)))
    if st != TACTKV_OK:
        raise TactkvError(st, "tactkv_occupancy")
    return {name: getattr(out, name) for name, _ in tactkv_occupancy_t._fields_}


def tactkv_max_batch(hbm_bytes: int, fixed_bytes: int, per_request_bytes: int) -> int:
    return int(_lib.tactkv_max_batch(int(hbm_bytes), int(fixed_bytes), int(per_request_bytes)))


def batch_capacity(hbm_bytes: int, fixed_bytes: int, payload_bytes_per_request: int, text_kv_bytes_per_request: int,
                   visual_kv_bf16_bytes_per_request: int) -> dict:
    """Decode batch that fits with the visual KV compressed versus kept in bf16 (the text KV stays
    bf16 either way), and the per-request cache shrink."""
    comp = payload_bytes_per_request + text_kv_bytes_per_request
    full = visual_kv_bf16_bytes_per_request + text_kv_bytes_per_request
    return {"batch_bf16": tactkv_max_batch(hbm_bytes, fixed_bytes, full),
            "batch_compressed": tactkv_max_batch(hbm_bytes, fixed_bytes, comp),
            "cache_shrink": full / comp if comp else float("inf")}


def tactkv_status_string(status: int) -> str:
    return _lib.tactkv_status_string(int(status)).decode()


def tactkv_lloyd_max_table(bits: int):
    """The library's own codebook: (levels, thresholds) as lists of floats (host only)."""
    L = 1 << bits
    lv = (ctypes.c_double * L)()
    th = (ctypes.c_double * max(1, L - 1))()
    n = _lib.tactkv_lloyd_max_table(bits, lv, th)
    if n != L:
        raise ValueError("bits must be 1..8")
    return list(lv), list(th)[:L - 1]


def tactkv_format_version() -> int:
    return int(_lib.tactkv_format_version())


def tactkv_last_launches() -> int:
    """Kernels launched by this thread's most recent compress / decompress call."""
    return int(_lib.tactkv_last_launches())


def _as_array(units):
    if isinstance(units, ctypes.Array):
        return units
    units = list(units)
    arr = (tactkv_unit * len(units))(*units)
    return arr


# ------------------------------------------------------------------------------ torch helpers ---
def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def make_units(x: Optional[torch.Tensor], S: int, H: int, W: int, bits: int, *, heads: int, head_dim: int,
               payload: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               layers: Optional[Sequence[int]] = None, kvs: Optional[Sequence[int]] = None,
               flags: int = 0, n_units: Optional[int] = None):
    """Descriptors for a batch laid out as [units, tokens, heads, head_dim] (strided views allowed).

    x is the compress input (or None for decompress), out the decompress output, payload a
    [units, capacity] uint8 tensor."""
    ref = x if x is not None else out
    U = ref.shape[0] if n_units is None else n_units
    arr = (tactkv_unit * U)()
    for i in range(U):
        u = arr[i]
        u.layer = int(layers[i]) if layers is not None else i
        u.kv = int(kvs[i]) if kvs is not None else 0
        u.S, u.H, u.W, u.heads, u.head_dim, u.bits, u.flags = S, H, W, heads, head_dim, bits, flags
        if x is not None:
            u.kv_in = x[i].data_ptr()
            u.token_stride, u.head_stride = x.stride(1), x.stride(2)
        if out is not None:
            u.kv_out = out[i].data_ptr()
            u.token_stride, u.head_stride = out.stride(1), out.stride(2)
        if payload is not None:
            u.payload = payload[i].data_ptr()
            u.payload_capacity = payload.shape[1]
    return arr


def payload_capacity(S: int, H: int, W: int, heads: int, head_dim: int, bits: int, flags: int = 0) -> int:
    u = tactkv_unit(S=S, H=H, W=W, heads=heads, head_dim=head_dim, bits=bits, flags=flags)
    cap = tactkv_payload_bytes(u)
    if cap == 0:
        raise TactkvError(TACTKV_UNSUPPORTED_SHAPE, "payload_capacity")
    return cap


def alloc_workspace(units, device) -> torch.Tensor:
    nbytes = tactkv_workspace_bytes(units)
    ws = torch.zeros(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + nbytes]


def compress(x: torch.Tensor, S: int, H: int, W: int, bits: int, *, layers=None, kvs=None, flags: int = 0,
             payload: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Compress x [units, S*H*W, heads, head_dim] (bf16, or fp32 with TACTKV_FP32_IO) on its device.
    Returns the [units, capacity] uint8 payload tensor (asynchronous on the stream)."""
    U, T, heads, D = x.shape
    if x.dtype == torch.float32:
        flags |= TACTKV_FP32_IO
    cap = payload_capacity(S, H, W, heads, D, bits, flags)
    if payload is None:
        payload = torch.empty((U, (cap + 15) // 16 * 16), dtype=torch.uint8, device=x.device)
    units = make_units(x, S, H, W, bits, heads=heads, head_dim=D, payload=payload, layers=layers, kvs=kvs,
                       flags=flags)
    if workspace is None:
        workspace = alloc_workspace(units, x.device)
    st = tactkv_compress(units, workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    if st != TACTKV_OK:
        raise TactkvError(st, "tactkv_compress")
    return payload


def decompress(payload: torch.Tensor, S: int, H: int, W: int, bits: int, *, heads: int, head_dim: int,
               layers=None, kvs=None, flags: int = 0, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
               check: bool = False) -> torch.Tensor:
    """Decompress [units, capacity] payloads into [units, S*H*W, heads, head_dim]."""
    U = payload.shape[0]
    if dtype == torch.float32:
        flags |= TACTKV_FP32_IO
    if out is None:
        out = torch.empty((U, S * H * W, heads, head_dim), dtype=dtype, device=payload.device)
    units = make_units(None, S, H, W, bits, heads=heads, head_dim=head_dim, payload=payload, out=out,
                       layers=layers, kvs=kvs, flags=flags, n_units=U)
    if workspace is None:
        workspace = alloc_workspace(units, payload.device)
    st = tactkv_decompress(units, workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    if st != TACTKV_OK:
        raise TactkvError(st, "tactkv_decompress")
    if check:
        ds = tactkv_device_status(workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
        if ds != TACTKV_OK:
            raise TactkvError(ds, "tactkv_decompress (device)")
    return out


def attention_decode(q: torch.Tensor, k_payload: torch.Tensor, v_payload: torch.Tensor, S: int, H: int, W: int,
                     bits: int, *, heads: int, head_dim: int, layers=None, flags: int = 0,
                     workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                     check: bool = False):
    """One decode step of attention over compressed K/V: q [units, q_heads, head_dim] float32 on the
    GPU, k_payload / v_payload [units, capacity] (compressed with kv 0 / 1).  Returns (out, m, l):
    out [units, q_heads, head_dim] = softmax(q K^T / sqrt(head_dim)) V over the visual tokens, m and
    l the scores' maximum and exp-sum per query head."""
    U, q_heads, D = q.shape
    q = q.contiguous().to(torch.float32)
    ku = make_units(None, S, H, W, bits, heads=heads, head_dim=head_dim, payload=k_payload, layers=layers,
                    kvs=[0] * U, flags=flags, n_units=U)
    vu = make_units(None, S, H, W, bits, heads=heads, head_dim=head_dim, payload=v_payload, layers=layers,
                    kvs=[1] * U, flags=flags, n_units=U)
    out = torch.empty((U, q_heads, D), dtype=torch.float32, device=q.device)
    m = torch.empty((U, q_heads), dtype=torch.float32, device=q.device)
    l = torch.empty((U, q_heads), dtype=torch.float32, device=q.device)
    if workspace is None:
        nbytes = tactkv_attention_workspace_bytes(ku, U, q_heads)
        ws = torch.zeros(nbytes + 256, dtype=torch.uint8, device=q.device)
        off = (-ws.data_ptr()) % 256
        workspace = ws[off:off + nbytes]
    st = int(_lib.tactkv_attention_decode(ku, vu, U, q_heads, ctypes.c_void_p(q.data_ptr()),
                                          ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(m.data_ptr()),
                                          ctypes.c_void_p(l.data_ptr()), ctypes.c_void_p(workspace.data_ptr()),
                                          workspace.numel(), ctypes.c_void_p(_stream_ptr(stream))))
    if st != TACTKV_OK:
        raise TactkvError(st, "tactkv_attention_decode")
    if check:
        ds = tactkv_device_status(workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
        if ds != TACTKV_OK:
            raise TactkvError(ds, "tactkv_attention_decode (device)")
    return out, m, l


# --------------------------------------------------------------------------------- text cache ---
class TextCache:
    """One layer's paged text K/V: the pools (uint8 tensors on one GPU) and their format.

    fmt "bf16", "mxfp8" or "mxfp4".  k_pages, v_pages [n_pages, heads, page_tokens, head_dim * 16, 8 or 4 / 8] hold
    the codes, k_scales, v_scales [n_pages, heads, page_tokens, head_dim / 32] the scale bytes (None
    with "bf16", whose pools may also be bfloat16 tensors [..., head_dim]).  text_cache() allocates them."""

    def __init__(self, fmt: str, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None):
        self.format = TEXT_FORMATS[fmt]
        if fmt == "bf16":
            k_pages, v_pages = (x.view(torch.uint8) if x.dtype == torch.bfloat16 else x for x in (k_pages, v_pages))
            k_scales = v_scales = None
        pools = [k_pages, v_pages] + ([] if fmt == "bf16" else [k_scales, v_scales])
        if any(x is None or x.dtype != torch.uint8 or not x.is_contiguous() or x.dim() != 4 or not x.is_cuda
               or x.device != k_pages.device for x in pools):
            raise ValueError("the text cache's pools are contiguous 4-D uint8 tensors on one GPU")
        self.n_pages, self.heads, self.page_tokens, row_bytes = k_pages.shape
        self.head_dim = row_bytes * 8 // (16, 8, 4)[self.format]
        if v_pages.shape != k_pages.shape or any(x.shape != (*k_pages.shape[:3], self.head_dim // 32)
                                                 for x in pools[2:]):
            raise ValueError("the text cache's pools do not fit together")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k_pages, v_pages, k_scales, v_scales
        self.device = k_pages.device
        self.struct = tactkv_text_cache(self.format, self.heads, self.head_dim, self.page_tokens, self.n_pages,
                                        *[x.data_ptr() for x in pools])
        self.ptr = ctypes.addressof(self.struct)
        if tactkv_text_workspace_bytes(self, 0, 0, 0, 0, 0) == 0:
            raise TactkvError(TACTKV_UNSUPPORTED_SHAPE, "TextCache")


def text_cache(fmt: str, n_pages: int, heads: int, head_dim: int, *, page_tokens: int = 64, device="cuda") -> TextCache:
    """A TextCache of zeroed pools."""
    row = head_dim * (16, 8, 4)[TEXT_FORMATS[fmt]] // 8
    shapes = [row, row] + ([] if fmt == "bf16" else [head_dim // 32] * 2)
    return TextCache(fmt, *[torch.zeros((n_pages, heads, page_tokens, w), dtype=torch.uint8, device=device) for w in shapes])


_INT_MAX = (1 << 31) - 1


def tactkv_text_workspace_bytes(cache: TextCache, n_seqs: int, n_rows: int, q_heads: int, max_rows: int,
                                max_kv_len: int) -> int:
    numbers = (n_seqs, n_rows, q_heads, max_rows, max_kv_len)
    if max(numbers) > _INT_MAX or min(numbers) < 0:   # ctypes would take them modulo 2^32
        return 0
    return int(_lib.tactkv_text_workspace_bytes(cache.ptr, *numbers))


def text_workspace(cache: TextCache, *, n_seqs: int, n_rows: int, max_rows: int = 1, q_heads: int = 0,
                   max_kv_len: int = 0) -> torch.Tensor:
    """Zeroed workspace for calls of up to these sizes (q_heads = 0: append and read alone)."""
    nbytes = tactkv_text_workspace_bytes(cache, n_seqs, n_rows, q_heads, max_rows, max_kv_len)
    if nbytes == 0:
        raise TactkvError(TACTKV_INVALID_ARG, "text_workspace")
    ws = torch.zeros(nbytes + 256, dtype=torch.uint8, device=cache.device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + nbytes]


def text_tree(parents: Sequence[Sequence[int]], device="cuda") -> torch.Tensor:
    """The tree words [rows] int64 of sequences whose drafted tokens hang under the given earlier ones:
    parents[s][j] < j is the parent of sequence s's node j, -1 for a root.  Bit i of a node's word is set
    for its ancestors and for itself."""
    words = []
    for seq in parents:
        mine = []
        for j, up in enumerate(seq):
            if not -1 <= up < j or j >= 64:
                raise ValueError("a node's parent is an earlier node of at most 64, or -1")
            mine.append((mine[up] if up >= 0 else 0) | 1 << j)
        words += [w - (1 << 64) if w >> 63 else w for w in mine]
    return torch.tensor(words, dtype=torch.int64, device=device)


_TEXT_BATCH = struct.Struct("@PPPiii")   # tactkv_text_batch
_TEXT_IO = {torch.bfloat16: 0, torch.float32: TACTKV_FP32_IO}


def _text_batch(cache: TextCache, page_table: torch.Tensor, kv_lens: torch.Tensor, row_starts: torch.Tensor,
                n_rows: int) -> bytes:
    n_seqs, max_pages = page_table.shape
    for x in (page_table, kv_lens, row_starts):
        if x.dtype != torch.int32 or not x.is_contiguous() or x.device != cache.device:
            raise ValueError("page_table, kv_lens and row_starts are contiguous int32 tensors on the cache's GPU")
    if kv_lens.numel() != n_seqs or row_starts.numel() != n_seqs + 1:
        raise ValueError("page_table [n_seqs, max_pages], kv_lens [n_seqs], row_starts [n_seqs + 1]")
    return _TEXT_BATCH.pack(page_table.data_ptr(), kv_lens.data_ptr(), row_starts.data_ptr(), n_seqs, n_rows, max_pages)


def _text_elsewhere(cache: TextCache, stream: Optional[torch.cuda.Stream]) -> bool:
    """Whether a call needs another device or stream made current first.  What it allocates and converts then
    belongs to the stream that it runs on."""
    return stream is not None or torch.cuda.current_device() != cache.device.index


def _text_there(cache: TextCache, stream: Optional[torch.cuda.Stream]):
    if stream is None:
        return torch.cuda.device(cache.device)
    if stream.device != cache.device:
        raise ValueError("the stream is not on the cache's GPU")
    return torch.cuda.stream(stream)


def _text_done(status: int, what: str, check: bool, workspace: torch.Tensor, stream_ptr: int) -> None:
    if status != TACTKV_OK:
        raise TactkvError(status, what)
    if check:
        ds = tactkv_device_status(workspace.data_ptr(), workspace.numel(), stream_ptr)
        if ds != TACTKV_OK:
            raise TactkvError(ds, what + " (device)")


def _text_pair(cache: TextCache, k: torch.Tensor, v: torch.Tensor, write: bool):
    """k and v [rows, heads, head_dim] with one pair of strides, as the library takes them: (k, v, strides)."""
    if (k.dtype not in _TEXT_IO or v.dtype != k.dtype or k.dim() != 3 or v.shape != k.shape
            or k.shape[1:] != (cache.heads, cache.head_dim) or k.device != cache.device or v.device != cache.device):
        raise ValueError("k and v [rows, heads, head_dim] are bfloat16 or float32 tensors on the cache's GPU")
    strides = k.stride()
    if (v.stride() != strides or strides[2] != 1 or strides[0] <= 0 or strides[0] % 2 or strides[1] % 2
            or (k.data_ptr() | v.data_ptr()) % (2 * k.element_size())):
        if write:
            raise ValueError("k and v start at an even element and have equal even strides, and neighbouring values along "
                             "head_dim")
        k, v = (x.clone(memory_format=torch.contiguous_format) for x in (k, v))
        strides = k.stride()
    return k, v, strides


def text_append(cache: TextCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                row_starts: torch.Tensor, *, values: bool = False, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None, check: bool = False):
    """Write k, v [rows, heads, head_dim] (bfloat16 or float32) into the cache: the rows row_starts[s] ..
    row_starts[s+1] are sequence s's newest tokens, at positions kv_lens[s] - n .. kv_lens[s] - 1 (kv_lens counts
    them).  page_table [n_seqs, max_pages], kv_lens and row_starts are int32 on the GPU.  k and v that do not start at an even
    element, or whose strides differ or are odd, are copied first.  With values, returns (k, v) as the cache now holds
    them (rows behind the last sequence are left unset)."""
    if _text_elsewhere(cache, stream):
        with _text_there(cache, stream):
            return text_append(cache, k, v, page_table, kv_lens, row_starts, values=values, workspace=workspace, check=check)
    k, v, strides = _text_pair(cache, k, v, False)
    batch = _text_batch(cache, page_table, kv_lens, row_starts, k.shape[0])
    out, kp, vp = None, None, None
    if values:
        out = (torch.empty_like(k, memory_format=torch.contiguous_format),
               torch.empty_like(v, memory_format=torch.contiguous_format))
        kp, vp = out[0].data_ptr(), out[1].data_ptr()
    if workspace is None:
        workspace = text_workspace(cache, n_seqs=0, n_rows=0)
    stream_ptr = torch._C._cuda_getCurrentRawStream(cache.device.index)
    st = _lib.tactkv_text_append(cache.ptr, batch, k.data_ptr(), v.data_ptr(), strides[0], strides[1], kp, vp,
                                 _TEXT_IO[k.dtype], workspace.data_ptr(), workspace.numel(), stream_ptr)
    if st or check:
        _text_done(st, "tactkv_text_append", check, workspace, stream_ptr)
    return out


def text_read(cache: TextCache, page_table: torch.Tensor, kv_lens: torch.Tensor, row_starts: torch.Tensor, *,
              n_rows: int, dtype=torch.bfloat16, out=None, workspace: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None, check: bool = False):
    """Read the newest row_starts[s+1] - row_starts[s] tokens of every sequence (all kv_lens[s] of them, if that is
    as many): (k, v) [n_rows, heads, head_dim], into the pair out if given (rows behind the last sequence are
    left as they are)."""
    if _text_elsewhere(cache, stream):
        with _text_there(cache, stream):
            return text_read(cache, page_table, kv_lens, row_starts, n_rows=n_rows, dtype=dtype, out=out,
                             workspace=workspace, check=check)
    if out is None:
        k = torch.empty(n_rows, cache.heads, cache.head_dim, dtype=dtype, device=cache.device)
        out = (k, torch.empty_like(k))
    k, v, strides = _text_pair(cache, out[0], out[1], True)
    if k.shape[0] != n_rows:
        raise ValueError("out holds n_rows rows")
    batch = _text_batch(cache, page_table, kv_lens, row_starts, n_rows)
    if workspace is None:
        workspace = text_workspace(cache, n_seqs=0, n_rows=0)
    stream_ptr = torch._C._cuda_getCurrentRawStream(cache.device.index)
    st = _lib.tactkv_text_read(cache.ptr, batch, k.data_ptr(), v.data_ptr(), strides[0], strides[1],
                               _TEXT_IO[k.dtype], workspace.data_ptr(), workspace.numel(), stream_ptr)
    if st or check:
        _text_done(st, "tactkv_text_read", check, workspace, stream_ptr)
    return out


def text_attention(q: torch.Tensor, cache: TextCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
                   row_starts: torch.Tensor, *, max_rows: int, max_kv_len: Optional[int] = None,
                   tree: Optional[torch.Tensor] = None, prior=None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                   check: bool = False):
    """Attention of the newest rows q [rows, q_heads, head_dim] (bfloat16 or float32) over their sequences' cached
    tokens, those rows' own among them: one generated token for each sequence (max_rows = 1), or up to 64
    drafted ones whose tree words (text_tree) say which of the others each sees (None: the ones before it).
    max_kv_len bounds kv_lens (default: what the page table holds).  prior = (out, m, l) merges the same
    queries' attention over other tokens, as attention_decode returns it (float32).  Returns (out, m, l): out
    like q; m and l float32 [rows, q_heads], the scores' maximum and exp-sum with the prior's.  Rows behind the last
    sequence are left as they are.  Without workspace (text_workspace) the call makes and zeroes its own, of 5 to 20 MB; what the
    kernels find wrong is in the workspace, and raised with check."""
    if not (0 <= max_rows <= _INT_MAX and (max_kv_len is None or 0 <= max_kv_len <= _INT_MAX)):
        raise TactkvError(TACTKV_INVALID_ARG, "tactkv_text_attention")
    if _text_elsewhere(cache, stream):
        with _text_there(cache, stream):
            return text_attention(q, cache, page_table, kv_lens, row_starts, max_rows=max_rows, max_kv_len=max_kv_len,
                                  tree=tree, prior=prior, out=out, workspace=workspace, check=check)
    device = cache.device
    shape = q.shape
    if q.dtype not in _TEXT_IO or len(shape) != 3 or shape[2] != cache.head_dim or q.device != device:
        raise ValueError("q [rows, q_heads, head_dim] is a bfloat16 or float32 tensor on the cache's GPU")
    n_rows, q_heads, D = shape
    strides = q.stride()
    if strides[2] != 1 or strides[0] % 8 or strides[1] % 8 or q.data_ptr() % 16:
        q = q.clone(memory_format=torch.contiguous_format)
        strides = q.stride()
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.shape != shape or out.dtype != q.dtype or not out.is_contiguous() or out.device != device:
        raise ValueError("out is a contiguous tensor of q's shape, type and device")
    m = torch.empty(n_rows, q_heads, dtype=torch.float32, device=device)
    l = torch.empty_like(m)
    tree_ptr = None
    if tree is not None:
        if tree.dtype != torch.int64 or tree.numel() != n_rows or not tree.is_contiguous() or tree.device != device:
            raise ValueError("tree holds an int64 word for each row")
        tree_ptr = tree.data_ptr()
    po = pm = pl = None
    if prior is not None:
        po, pm, pl = prior
        if (po.shape != shape or pm.shape != m.shape or pl.shape != m.shape
                or any(x.dtype != torch.float32 or not x.is_contiguous() or x.device != device for x in prior)):
            raise ValueError("prior = (out, m, l): contiguous float32 [rows, q_heads, head_dim], [rows, q_heads] (twice)")
        po, pm, pl = po.data_ptr(), pm.data_ptr(), pl.data_ptr()
    batch = _text_batch(cache, page_table, kv_lens, row_starts, n_rows)
    if max_kv_len is None:
        max_kv_len = min(page_table.shape[1] * cache.page_tokens, 1 << 30)
    if workspace is None:
        workspace = text_workspace(cache, n_seqs=page_table.shape[0], n_rows=n_rows, max_rows=max_rows, q_heads=q_heads,
                                   max_kv_len=max_kv_len)
    stream_ptr = torch._C._cuda_getCurrentRawStream(device.index)
    st = _lib.tactkv_text_attention(cache.ptr, batch, q_heads, max_rows, max_kv_len, q.data_ptr(), strides[0],
                                    strides[1], tree_ptr, po, pm, pl, out.data_ptr(), m.data_ptr(), l.data_ptr(),
                                    _TEXT_IO[q.dtype], workspace.data_ptr(), workspace.numel(), stream_ptr)
    if st or check:
        _text_done(st, "tactkv_text_attention", check, workspace, stream_ptr)
    return out, m, l
