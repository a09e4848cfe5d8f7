"""B200 (sm_100a) decode attention over a K8/V4-quantised, segmented KV cache.

Thin Python binding of ``libnf.so`` (the C ABI declared in ``include/nf.h``):
appending, decode and prefill attention, and for sessions that bound their
context the windowed forms, rotary positions on the way into the cache and the
pages of the pool.
Every function here only marshals torch tensors into pointers and sizes and
calls the C entry point of the same name; all computation happens in the CUDA
kernels of ``csrc/``.  torch provides device memory and the current stream.
There is no CPU fallback: if ``libnf.so`` is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

import torch

__all__ = [
    "NF_OK", "NF_KV_K8V4", "NF_KV_BF16", "NF_KV_K8V8", "NF_KV_F8", "NF_KV_K4V4", "NF_F32", "NF_BF16", "NfError", "KVLayer",
    "nf_kv_append_quant", "nf_decode_attn_workspace_size", "nf_decode_attn", "nf_decode_attn_noalloc",
    "nf_attn_combine", "nf_attn_packed_slot_floats", "nf_attn_combine_packed", "nf_prefill_attn",
    "nf_decode_attn_window", "nf_decode_attn_window_workspace_size", "nf_prefill_attn_window",
    "Rope", "NF_ROPE_HALVES", "NF_ROPE_PAIRS", "nf_rope_append_quant",
    "KVLayers", "nf_kv_reserve", "nf_kv_release", "nf_kv_copy_blocks", "nf_kv_pages_workspace_size", "nf_kv_fork",
    "nf_kv_compact",
    "nf_get_device_error", "nf_status_string", "library_path", "load_library",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
HEADER = os.path.join(_ROOT, "include", "nf.h")
_LIB_PATH = os.path.join(_PKG, "libnf.so")

NF_OK = 0
NF_ERR_INVALID_ARG, NF_ERR_UNSUPPORTED, NF_ERR_WORKSPACE, NF_ERR_CUDA, NF_ERR_DEVICE_CHECK = 1, 2, 3, 4, 5
NF_DEVERR_NONE, NF_DEVERR_BLOCK_ID, NF_DEVERR_TABLE, NF_DEVERR_SEQLEN = 0, 1, 2, 3
NF_DEVERR_TIMEOUT, NF_DEVERR_INTERNAL, NF_DEVERR_RANGE = 4, 5, 6
NF_DEVERR_CONFLICT, NF_DEVERR_POOL, NF_DEVERR_REFS = 7, 8, 9
NF_ROPE_HALVES, NF_ROPE_PAIRS, NF_ROPE_MAX_AXES = 0, 1, 4
NF_F32, NF_BF16, NF_F16 = 0, 1, 2
NF_KV_K8V4, NF_KV_BF16, NF_KV_K8V8, NF_KV_F8, NF_KV_K4V4 = 0, 1, 2, 3, 4
BLOCK = 256
HEAD_DIM = 128


class NfError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {message} (status {status})")
        self.status = status


class nf_kv_layer(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int32), ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("v_group", ctypes.c_int32),
        ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
    ]


class nf_rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("axis", ctypes.c_uint8 * 64), ("inv_freq", ctypes.c_void_p)]


class nf_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


_pack_q_k_v = struct.Struct("@PqqPqqPqq").pack  # three nf_heads, without building ctypes objects


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libnf.so (built by ``python -m long_context_quantized_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: build it with "
                              "`python -m long_context_quantized_b200.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        lib.nf_kv_append_quant.argtypes = [P, P, P, I, I, I, P, I, P, P]
        lib.nf_kv_append_quant.restype = I
        lib.nf_decode_attn_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.nf_decode_attn_workspace_size.restype = S
        lib.nf_decode_attn.argtypes = [P, P, I, I, I, I, P, I, P, I, ctypes.c_float, I, P, P, P, S, P]
        lib.nf_decode_attn.restype = I
        lib.nf_decode_attn_ex.argtypes = [P, P, I, I, I, I, P, I, P, I, ctypes.c_float, I, ctypes.c_uint32, P, P,
                                          P, S, P]
        lib.nf_decode_attn_ex.restype = I
        lib.nf_decode_attn_noalloc.argtypes = [P, P, I, I, I, I, P, I, P, I, ctypes.c_float, I, P, P, P]
        lib.nf_decode_attn_noalloc.restype = I
        lib.nf_prefill_attn.argtypes = [P, P, I, I, I, I, P, I, P, I, ctypes.c_float, I, P, P, P]
        lib.nf_prefill_attn.restype = I
        lib.nf_selftest_bounded_wait.argtypes = [ctypes.c_uint32, P]
        lib.nf_selftest_bounded_wait.restype = I
        lib.nf_attn_combine.argtypes = [P, P, I, I, I, P, P, P]
        lib.nf_attn_combine.restype = I
        lib.nf_attn_packed_slot_floats.argtypes = [I, I]
        lib.nf_attn_packed_slot_floats.restype = S
        lib.nf_attn_combine_packed.argtypes = [P, I, I, I, P, P, P]
        lib.nf_attn_combine_packed.restype = I
        F = ctypes.c_float
        lib.nf_decode_attn_window_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.nf_decode_attn_window_workspace_size.restype = S
        lib.nf_decode_attn_window.argtypes = [P, P, I, I, I, I, P, I, P, I, I, I, F, P, I, P, P, S, P]
        lib.nf_decode_attn_window.restype = I
        lib.nf_prefill_attn_window.argtypes = [P, P, I, I, I, I, P, I, P, I, I, I, F, P, I, P, P]
        lib.nf_prefill_attn_window.restype = I
        lib.nf_rope_append_quant.argtypes = [P, P, P, P, I, I, I, I, P, I, P, P, P, P]
        lib.nf_rope_append_quant.restype = I
        lib.nf_kv_reserve.argtypes = lib.nf_kv_release.argtypes = [P, I, P, I, I, P, P, P]
        lib.nf_kv_reserve.restype = lib.nf_kv_release.restype = I
        lib.nf_kv_copy_blocks.argtypes = [P, I, P, P, I, P]
        lib.nf_kv_copy_blocks.restype = I
        lib.nf_kv_pages_workspace_size.argtypes = [I, I]
        lib.nf_kv_pages_workspace_size.restype = S
        lib.nf_kv_fork.argtypes = [P, I, P, P, I, I, P, P, I, P, P, S, P]
        lib.nf_kv_fork.restype = I
        lib.nf_kv_compact.argtypes = [P, I, P, P, I, I, P, S, P]
        lib.nf_kv_compact.restype = I
        lib.nf_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_int32)]
        lib.nf_get_device_error.restype = I
        lib.nf_status_string.argtypes = [I]
        lib.nf_status_string.restype = ctypes.c_char_p
        lib.nf_last_error.argtypes = []
        lib.nf_last_error.restype = ctypes.c_char_p
        _lib = lib
        return lib


def declared_symbols(header: str = HEADER) -> list:
    """Names of the functions include/nf.h declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(nf_[a-z_0-9]+)\s*\(", text)))


def _check(st: int, where: str):
    if st != NF_OK:
        lib = load_library()
        raise NfError(st, where, lib.nf_last_error().decode() or lib.nf_status_string(st).decode())


def _int32(where: str, *values):
    """Refuses integers that ctypes would cut to their low 32 bits."""
    for v in values:
        if not -0x80000000 <= v <= 0x7FFFFFFF:
            raise NfError(NF_ERR_INVALID_ARG, where, f"{v} is outside the range of a 32-bit integer")


def _dptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_current_device = torch.cuda.current_device


def _raw_stream(device: int) -> int:
    # looked up at the call: a torch built without CUDA lacks it, and imports this package for its host logic
    return torch._C._cuda_getCurrentRawStream(device)


def _stream(stream):
    if stream is None:  # the current stream's handle, without building a Stream object
        return _raw_stream(_current_device())
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return NF_F32
    if dt == torch.bfloat16:
        return NF_BF16
    raise NfError(NF_ERR_UNSUPPORTED, "dtype", f"{dt} (float32 or bfloat16)")


def _need(t, name, dtype=None, device=True):
    if t is None:
        return
    if not t.is_contiguous():
        raise NfError(NF_ERR_INVALID_ARG, name, "tensor must be contiguous")
    if device and not t.is_cuda:
        raise NfError(NF_ERR_INVALID_ARG, name, "tensor must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise NfError(NF_ERR_INVALID_ARG, name, f"dtype {t.dtype}, expected {dtype}")


class KVLayer:
    """One layer's KV pool planes (device tensors owned by torch) and the
    ``nf_kv_layer`` view the C ABI takes.  Layout: see ``include/nf.h``."""

    def __init__(self, fmt: int, k_codes, k_scales, v_codes, v_scales):
        self.fmt = fmt
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.num_blocks, self.num_kv_heads = k_codes.shape[0], k_codes.shape[1]
        self.c = nf_kv_layer(fmt, self.num_blocks, BLOCK, self.num_kv_heads, HEAD_DIM, 32,
                             k_codes.data_ptr(), 0 if k_scales is None else k_scales.data_ptr(),
                             v_codes.data_ptr(), 0 if v_scales is None else v_scales.data_ptr())
        self.ref = ctypes.byref(self.c)
        self.device = k_codes.get_device()

    @classmethod
    def empty(cls, fmt: int, num_blocks: int, num_kv_heads: int, device="cuda", fill: int | None = None):
        kw = dict(device=device)
        if fmt == NF_KV_K8V4:
            k = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM), dtype=torch.int8, **kw)
            ks = torch.empty((num_blocks, num_kv_heads, BLOCK), dtype=torch.float16, **kw)
            v = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM // 2), dtype=torch.uint8, **kw)
            vs = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM // 32), dtype=torch.float16, **kw)
        elif fmt == NF_KV_K4V4:
            k = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM // 2), dtype=torch.uint8, **kw)
            ks = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM // 32), dtype=torch.uint8, **kw)
            v = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM // 2), dtype=torch.uint8, **kw)
            vs = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM // 32), dtype=torch.uint8, **kw)
        elif fmt in (NF_KV_K8V8, NF_KV_F8):
            code = torch.int8 if fmt == NF_KV_K8V8 else torch.uint8  # fp8: e4m3 bytes
            k = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM), dtype=code, **kw)
            ks = torch.empty((num_blocks, num_kv_heads, BLOCK), dtype=torch.float16, **kw)
            v = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM), dtype=code, **kw)
            vs = torch.empty((num_blocks, num_kv_heads, BLOCK), dtype=torch.float16, **kw)
        elif fmt == NF_KV_BF16:
            k = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM), dtype=torch.bfloat16, **kw)
            v = torch.empty((num_blocks, num_kv_heads, BLOCK, HEAD_DIM), dtype=torch.bfloat16, **kw)
            ks = vs = None
        else:
            raise NfError(NF_ERR_UNSUPPORTED, "KVLayer.empty", f"fmt {fmt}")
        if fill is not None:
            for t in (k, ks, v, vs):
                if t is not None:
                    t.view(torch.uint8).fill_(fill)
        return cls(fmt, k, ks, v, vs)

    def planes(self):
        return [t for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales) if t is not None]

    def bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.planes())


def nf_kv_append_quant(kv: KVLayer, k_new, v_new, block_table, seqlens_before, stream=None):
    """Quantise k_new / v_new [batch][n_new][H_kv][128] (fp32 or bf16) into the
    pool at positions seqlens_before[b] + i (see nf.h)."""
    _need(k_new, "k_new")
    _need(v_new, "v_new", k_new.dtype)
    _need(block_table, "block_table", torch.int32)
    _need(seqlens_before, "seqlens_before", torch.int32)
    B, n_new = k_new.shape[0], k_new.shape[1]
    st = load_library().nf_kv_append_quant(
        ctypes.byref(kv.c), _dptr(k_new), _dptr(v_new), _dtype_code(k_new.dtype), B, n_new,
        _dptr(block_table), block_table.shape[1], _dptr(seqlens_before), _stream(stream))
    _check(st, "nf_kv_append_quant")


def nf_decode_attn_workspace_size(batch, n_q, num_q_heads, num_kv_heads, max_seqlen, num_sms=None):
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    _int32("nf_decode_attn_workspace_size", batch, n_q, num_q_heads, num_kv_heads, max_seqlen, num_sms)
    return int(load_library().nf_decode_attn_workspace_size(batch, n_q, num_q_heads, num_kv_heads,
                                                            max_seqlen, num_sms))


NF_DECODE_EARLY_KV = 1


def nf_decode_attn(kv: KVLayer, q, block_table, seqlens, max_seqlen: int, softmax_scale: float,
                   causal: bool, out, out_lse=None, workspace=None, stream=None):
    """Decode attention; q [batch][n_q][H_q][128] (fp32 or bf16), out fp32 of
    the same shape, out_lse fp32 [batch][n_q][H_q] or None (see nf.h)."""
    nf_decode_attn_ex(kv, q, block_table, seqlens, max_seqlen, softmax_scale, causal, 0, out, out_lse,
                      workspace, stream, _name="nf_decode_attn")


def nf_decode_attn_ex(kv: KVLayer, q, block_table, seqlens, max_seqlen: int, softmax_scale: float,
                      causal: bool, flags: int, out, out_lse=None, workspace=None, stream=None,
                      _name="nf_decode_attn_ex"):
    """nf_decode_attn with flags (NF_DECODE_EARLY_KV: see nf.h for the caller's
    guarantee)."""
    _int32(_name, max_seqlen, flags)
    _need(q, "q")
    _need(block_table, "block_table", torch.int32)
    _need(seqlens, "seqlens", torch.int32)
    _need(out, "out", torch.float32)
    _need(out_lse, "out_lse", torch.float32)
    _need(workspace, "workspace")
    B, n_q, H_q = q.shape[0], q.shape[1], q.shape[2]
    if workspace is None:
        raise NfError(NF_ERR_WORKSPACE, _name, "workspace tensor required "
                      "(size: nf_decode_attn_workspace_size)")
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load_library().nf_decode_attn_ex(
        ctypes.byref(kv.c), _dptr(q), _dtype_code(q.dtype), B, n_q, H_q, _dptr(block_table),
        block_table.shape[1], _dptr(seqlens), int(max_seqlen), float(softmax_scale), int(bool(causal)),
        int(flags), _dptr(out), _dptr(out_lse), _dptr(workspace), ws_bytes, _stream(stream))
    _check(st, _name)


def nf_prefill_attn(kv: KVLayer, q, block_table, seqlens, max_seqlen: int, softmax_scale: float,
                    causal: bool, out, out_lse=None, stream=None):
    """Chunked-prefill attention (see nf.h): the n_q queries of each sequence
    at positions L - n_q .. L - 1 against its K8/V4 cache; q bf16
    [batch][n_q][H_q][128], out fp32 of the same shape."""
    _int32("nf_prefill_attn", max_seqlen)
    _need(q, "q")
    _need(block_table, "block_table", torch.int32)
    _need(seqlens, "seqlens", torch.int32)
    _need(out, "out", torch.float32)
    _need(out_lse, "out_lse", torch.float32)
    B, n_q, H_q = q.shape[0], q.shape[1], q.shape[2]
    st = load_library().nf_prefill_attn(
        ctypes.byref(kv.c), _dptr(q), _dtype_code(q.dtype), B, n_q, H_q, _dptr(block_table),
        block_table.shape[1], _dptr(seqlens), int(max_seqlen), float(softmax_scale), int(bool(causal)),
        _dptr(out), _dptr(out_lse), _stream(stream))
    _check(st, "nf_prefill_attn")


NF_NOALLOC_SCRATCH_BYTES = 8 << 20


def nf_decode_attn_noalloc(kv: KVLayer, q, block_table, seqlens, max_seqlen: int, softmax_scale: float,
                           causal: bool, out, out_lse=None, stream=None):
    """nf_decode_attn for callers that cannot allocate device memory at call
    time: the scratch is a fixed array inside libnf's device image (see nf.h).
    Calls on one device share it, so do not overlap them on the GPU."""
    _int32("nf_decode_attn_noalloc", max_seqlen)
    _need(q, "q")
    _need(block_table, "block_table", torch.int32)
    _need(seqlens, "seqlens", torch.int32)
    _need(out, "out", torch.float32)
    _need(out_lse, "out_lse", torch.float32)
    B, n_q, H_q = q.shape[0], q.shape[1], q.shape[2]
    st = load_library().nf_decode_attn_noalloc(
        ctypes.byref(kv.c), _dptr(q), _dtype_code(q.dtype), B, n_q, H_q, _dptr(block_table),
        block_table.shape[1], _dptr(seqlens), int(max_seqlen), float(softmax_scale), int(bool(causal)),
        _dptr(out), _dptr(out_lse), _stream(stream))
    _check(st, "nf_decode_attn_noalloc")


def nf_attn_combine(part_o, part_lse, out, out_lse=None, stream=None):
    """part_o [S][rows][d], part_lse [S][rows] (fp32) -> out [rows][d], out_lse [rows]."""
    _need(part_o, "part_o", torch.float32)
    _need(part_lse, "part_lse", torch.float32)
    _need(out, "out", torch.float32)
    _need(out_lse, "out_lse", torch.float32)
    S, rows, d = part_o.shape
    st = load_library().nf_attn_combine(_dptr(part_o), _dptr(part_lse), S, rows, d, _dptr(out),
                                        _dptr(out_lse), _stream(stream))
    _check(st, "nf_attn_combine")


def nf_attn_packed_slot_floats(rows: int, head_dim: int = HEAD_DIM) -> int:
    """Floats of one packed split slot: o [rows][head_dim] then lse [rows],
    rounded up to a multiple of 4 (see nf.h)."""
    _int32("nf_attn_packed_slot_floats", rows, head_dim)
    return int(load_library().nf_attn_packed_slot_floats(int(rows), int(head_dim)))


def nf_attn_combine_packed(parts, rows: int, out, out_lse=None, stream=None):
    """parts fp32 [S][slot] (packed split slots) -> out [rows][d], out_lse [rows]."""
    _int32("nf_attn_combine_packed", rows)
    _need(parts, "parts", torch.float32)
    _need(out, "out", torch.float32)
    _need(out_lse, "out_lse", torch.float32)
    S = parts.shape[0]
    d = out.shape[-1]
    if parts.numel() != S * nf_attn_packed_slot_floats(rows, d):
        raise NfError(NF_ERR_INVALID_ARG, "nf_attn_combine_packed", "parts is not [S][slot]")
    st = load_library().nf_attn_combine_packed(_dptr(parts), S, int(rows), d, _dptr(out), _dptr(out_lse),
                                               _stream(stream))
    _check(st, "nf_attn_combine_packed")


def nf_get_device_error() -> int:
    """Read and clear the device error code (synchronises the device)."""
    code = ctypes.c_int32(0)
    st = load_library().nf_get_device_error(ctypes.byref(code))
    if st not in (NF_OK, NF_ERR_DEVICE_CHECK):
        _check(st, "nf_get_device_error")
    return code.value


def nf_status_string(status: int) -> str:
    return load_library().nf_status_string(int(status)).decode()


def nf_selftest_bounded_wait(limit_us: int, stream=None):
    """Run the bounded-wait self-test (see nf.h); afterwards
    nf_get_device_error() returns NF_DEVERR_TIMEOUT."""
    _int32("nf_selftest_bounded_wait", limit_us)
    _check(load_library().nf_selftest_bounded_wait(int(limit_us), _stream(stream)), "nf_selftest_bounded_wait")


# ---------------------------------------------------------------- windowed sessions
def _refuse(where, message):
    raise NfError(NF_ERR_INVALID_ARG, where, message)


# The checks below run at every call: a call's host time is most of what a
# short kernel costs its caller, so the good case is a few comparisons and what
# was wrong is worked out only then.
_i32 = torch.int32


def _bad(where, name, t, dtype, device):
    _refuse(where, f"{name}: {t.dtype} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}; "
                   f"expected a contiguous {dtype} tensor on cuda:{device}")


def _current(where, t) -> int:
    """The device number of t, which must be the current CUDA device."""
    d = t.get_device()
    if d < 0:
        _refuse(where, "tensors must be on a CUDA device")
    if d != _current_device():
        _refuse(where, f"tensors are on cuda:{d}, the current device is cuda:{_current_device()}")
    return d


def _on(where, name, t, device: int, dtype):
    """t must be contiguous, of dtype, on the device."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _bad(where, name, t, dtype, device)


def _vector(where, name, t, device: int, n: int) -> int:
    """The address of t, which must be contiguous int32 [n] on the device."""
    if t.dtype is not _i32 or t.get_device() != device or t.shape != (n,) or not t.is_contiguous():
        if t.dim() != 1 or len(t) != n:
            _refuse(where, f"{name}: {tuple(t.shape)}, expected [{n}]")
        _bad(where, name, t, _i32, device)
    return t.data_ptr()


def _call_stream(stream, device: int):
    return _raw_stream(device) if stream is None else _stream(stream)


def nf_decode_attn_window_workspace_size(batch, n_q, num_q_heads, num_kv_heads, max_seqlen, num_sms=None):
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    _int32("nf_decode_attn_window_workspace_size", batch, n_q, num_q_heads, num_kv_heads, max_seqlen, num_sms)
    return int(load_library().nf_decode_attn_window_workspace_size(batch, n_q, num_q_heads, num_kv_heads, max_seqlen,
                                                                   num_sms))


def _window_args(where, kv, q, block_table, seqlens, out, out_lse):
    """Checks what both windowed calls take; returns q's shape, the device and addresses."""
    d = _current(where, q)
    shape = q.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM or not q.is_contiguous():
        _refuse(where, "q must be contiguous [batch][n_q][H_q][128]")
    B = shape[0]
    if block_table.dtype is not _i32 or block_table.get_device() != d or not block_table.is_contiguous():
        _bad(where, "block_table", block_table, _i32, d)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        _refuse(where, "block_table must be [batch][max_blocks] with q's batch")
    if out.get_device() != d or out.shape != shape or not out.is_contiguous():
        _refuse(where, f"out must be contiguous, of q's shape, on cuda:{d}")
    if kv.device != d:
        _refuse(where, f"the pool is on cuda:{kv.device}, q on cuda:{d}")
    lse = None
    if out_lse is not None:
        _on(where, "out_lse", out_lse, d, torch.float32)
        if out_lse.shape != shape[:3]:
            _refuse(where, "out_lse must be [batch][n_q][H_q]")
        lse = out_lse.data_ptr()
    return shape, d, _vector(where, "seqlens", seqlens, d, B), lse


def nf_decode_attn_window(kv: KVLayer, q, block_table, seqlens, max_seqlen: int, window: int, n_sink: int,
                          softmax_scale: float, out, out_lse=None, workspace=None, stream=None):
    """Decode attention with a sliding window and sinks: a query at position P
    sees the keys t <= P with t > P - window or t < n_sink (see nf.h).  out
    (fp32 or bf16) has the shape of q [batch][n_q][H_q][128]; seqlens 0 marks an
    unused row of the batch."""
    _int32("nf_decode_attn_window", max_seqlen, window, n_sink)
    (B, n_q, H_q, _), d, lens, lse = _window_args("nf_decode_attn_window", kv, q, block_table, seqlens, out, out_lse)
    if workspace is None:
        raise NfError(NF_ERR_WORKSPACE, "nf_decode_attn_window", "workspace tensor required "
                      "(size: nf_decode_attn_window_workspace_size)")
    if workspace.get_device() != d or not workspace.is_contiguous():
        _bad("nf_decode_attn_window", "workspace", workspace, workspace.dtype, d)
    st = (_lib or load_library()).nf_decode_attn_window(
        kv.ref, q.data_ptr(), _dtype_code(q.dtype), B, n_q, H_q, block_table.data_ptr(), block_table.shape[1], lens,
        max_seqlen, window, n_sink, softmax_scale, out.data_ptr(), _dtype_code(out.dtype), lse, workspace.data_ptr(),
        workspace.nbytes, _call_stream(stream, d))
    if st:
        _check(st, "nf_decode_attn_window")


def nf_prefill_attn_window(kv: KVLayer, q, block_table, seqlens, max_seqlen: int, window: int, n_sink: int,
                           softmax_scale: float, out, out_lse=None, stream=None):
    """Chunked-prefill attention with a sliding window and sinks (see nf.h and
    nf_decode_attn_window): bf16 q over a K8/V4 pool, out fp32 or bf16."""
    _int32("nf_prefill_attn_window", max_seqlen, window, n_sink)
    (B, n_q, H_q, _), d, lens, lse = _window_args("nf_prefill_attn_window", kv, q, block_table, seqlens, out, out_lse)
    st = (_lib or load_library()).nf_prefill_attn_window(
        kv.ref, q.data_ptr(), _dtype_code(q.dtype), B, n_q, H_q, block_table.data_ptr(), block_table.shape[1], lens,
        max_seqlen, window, n_sink, softmax_scale, out.data_ptr(), _dtype_code(out.dtype), lse, _call_stream(stream, d))
    if st:
        _check(st, "nf_prefill_attn_window")


class Rope:
    """The rotary frequencies of a model: ``inv_freq`` (fp32 [rot_dim / 2],
    device), the position axis of each frequency (``axis``, a sequence of
    rot_dim / 2 numbers below ``n_axes``; None: axis 0 for all) and the layout
    of the channel pairs (see nf_rope in nf.h)."""

    def __init__(self, inv_freq, axis=None, n_axes: int = 1, layout: int = NF_ROPE_HALVES):
        _int32("Rope", n_axes, layout)
        _need(inv_freq, "inv_freq", torch.float32)
        half = inv_freq.numel()
        axis = [0] * half if axis is None else [int(a) for a in axis]
        if len(axis) != half or half > 64 or any(not 0 <= a < n_axes for a in axis):
            _refuse("Rope", "axis must hold one axis below n_axes for each of the (at most 64) frequencies")
        self.inv_freq, self.n_axes, self.device = inv_freq, int(n_axes), inv_freq.get_device()
        self.c = nf_rope(2 * half, layout, n_axes, (ctypes.c_uint8 * 64)(*axis), inv_freq.data_ptr())
        self.ref = ctypes.byref(self.c)


def _heads(where, name, t, dtype, device, shape):
    """Address, batch and token stride of t [batch][n_new][heads][128], whose heads must be contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _refuse(where, f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, expected {dtype} {shape} on cuda:{device}")
    sb, st, sh, sc = t.stride()
    if (sc != 1 or (sh != HEAD_DIM and shape[2] > 1)) and t.numel():
        _refuse(where, f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), sb, st


def nf_rope_append_quant(kv: KVLayer, rope: Rope, positions, q, k_new, v_new, block_table, seqlens_before, q_out,
                         n_valid=None, stream=None):
    """Turn q and k_new by the rotary angles of ``positions`` (int32
    [batch][n_new][n_axes]), write q_out, and quantise the turned keys and the
    values into the pool at seqlens_before[b] + i (see nf.h).  q [batch][n_new]
    [H_q][128], k_new and v_new [batch][n_new][H_kv][128] of one dtype may be
    strided views (of a fused projection's output) whose heads are contiguous;
    tokens from n_valid[b] on are padding.  q and q_out may be None."""
    where = "nf_rope_append_quant"
    d = _current(where, k_new)
    if k_new.dim() != 4:
        _refuse(where, "k_new must be [batch][n_new][H_kv][128]")
    B, n_new = k_new.shape[:2]
    dtype = k_new.dtype
    shape = (B, n_new, kv.num_kv_heads, HEAD_DIM)
    k = _heads(where, "k_new", k_new, dtype, d, shape)
    v = _heads(where, "v_new", v_new, dtype, d, shape)
    if q is not None:
        H_q = q.shape[2] if q.dim() == 4 else 0
        qh = _heads(where, "q", q, dtype, d, (B, n_new, H_q, HEAD_DIM))
        if q_out is None or q_out.shape != q.shape:
            _refuse(where, "q_out must have q's shape")
        _on(where, "q_out", q_out, d, dtype)
        out = q_out.data_ptr()
    else:
        H_q, qh, out = 0, (0, 0, 0), None
    _on(where, "positions", positions, d, _i32)
    _on(where, "block_table", block_table, d, _i32)
    if kv.device != d or rope.device != d:
        _refuse(where, "the pool, inv_freq and the inputs must be on one device")
    if positions.shape != (B, n_new, rope.n_axes):
        _refuse(where, f"positions must be [batch][n_new][{rope.n_axes}]")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        _refuse(where, "block_table must be [batch][max_blocks] with the inputs' batch")
    st = (_lib or load_library()).nf_rope_append_quant(
        kv.ref, rope.ref, positions.data_ptr(), _pack_q_k_v(*qh, *k, *v), _dtype_code(dtype), B, n_new, H_q,
        block_table.data_ptr(), block_table.shape[1], _vector(where, "seqlens_before", seqlens_before, d, B),
        None if n_valid is None else _vector(where, "n_valid", n_valid, d, B), out, _call_stream(stream, d))
    if st:
        _check(st, where)


class KVLayers:
    """The layers of one pool (KVLayer views of one format, block count and
    head count), for the page calls that move blocks in all of them."""

    def __init__(self, layers):
        self.layers = list(layers)
        if not self.layers:
            _refuse("KVLayers", "no layers")
        self.num_blocks, self.device = self.layers[0].num_blocks, self.layers[0].device
        if any(layer.device != self.device for layer in self.layers):
            _refuse("KVLayers", "the layers must be on one device")
        self.c = (nf_kv_layer * len(self.layers))(*[layer.c for layer in self.layers])

    def __len__(self):
        return len(self.layers)


def _pages_args(where, refs, block_table) -> int:
    d = _current(where, refs)
    _on(where, "refs", refs, d, _i32)
    _on(where, "block_table", block_table, d, _i32)
    if refs.dim() != 1 or block_table.dim() != 2:
        _refuse(where, "refs must be [num_blocks], block_table [rows][max_blocks]")
    return d


def _pool_args(where, layers, refs, block_table, workspace) -> int:
    d = _pages_args(where, refs, block_table)
    if refs.shape[0] != layers.num_blocks or layers.device != d:
        _refuse(where, "refs must have one count per block of the pool, on its device")
    _on(where, "workspace", workspace, d, workspace.dtype)
    return d


def _range_call(where, call, refs, block_table, from_pos, to_pos, stream):
    d = _pages_args(where, refs, block_table)
    rows, width = block_table.shape
    st = call(refs.data_ptr(), refs.shape[0], block_table.data_ptr(), rows, width,
              _vector(where, "from_pos", from_pos, d, rows), _vector(where, "to_pos", to_pos, d, rows),
              _call_stream(stream, d))
    if st:
        _check(st, where)


def nf_kv_reserve(refs, block_table, from_pos, to_pos, stream=None):
    """Fresh pages for the positions [from_pos[b], to_pos[b]) of every table
    row that have none (see nf.h): the lowest free blocks, in row order."""
    _range_call("nf_kv_reserve", (_lib or load_library()).nf_kv_reserve, refs, block_table, from_pos, to_pos, stream)


def nf_kv_release(refs, block_table, from_pos, to_pos, stream=None):
    """Give up the pages wholly inside [from_pos[b], to_pos[b]) of every table
    row (see nf.h): behind a window, or a whole sequence."""
    _range_call("nf_kv_release", (_lib or load_library()).nf_kv_release, refs, block_table, from_pos, to_pos, stream)


def nf_kv_copy_blocks(layers: KVLayers, src, dst, stream=None):
    """Copy block src[i] to dst[i] in every layer (int32 [n]; see nf.h)."""
    where = "nf_kv_copy_blocks"
    d = _current(where, src)
    if layers.device != d:
        _refuse(where, f"the pool is on cuda:{layers.device}, src on cuda:{d}")
    n = len(src) if src.dim() == 1 else -1
    st = (_lib or load_library()).nf_kv_copy_blocks(layers.c, len(layers), _vector(where, "src", src, d, n),
                                                    _vector(where, "dst", dst, d, n), n, _call_stream(stream, d))
    if st:
        _check(st, where)


def nf_kv_pages_workspace_size(num_blocks: int, n_forks: int = 0) -> int:
    """Bytes of workspace of nf_kv_fork (n_forks pairs) and nf_kv_compact."""
    _int32("nf_kv_pages_workspace_size", num_blocks, n_forks)
    return int(load_library().nf_kv_pages_workspace_size(num_blocks, n_forks))


def nf_kv_fork(layers: KVLayers, refs, block_table, src_rows, dst_rows, seqlens, workspace, stream=None):
    """Make table row dst_rows[i] a copy of row src_rows[i] (see nf.h): full
    pages are shared, a partly filled last page is copied in every layer, and
    seqlens[dst] = seqlens[src]."""
    where = "nf_kv_fork"
    d = _pool_args(where, layers, refs, block_table, workspace)
    rows, width = block_table.shape
    n = len(src_rows) if src_rows.dim() == 1 else -1
    st = (_lib or load_library()).nf_kv_fork(
        layers.c, len(layers), refs.data_ptr(), block_table.data_ptr(), rows, width,
        _vector(where, "src_rows", src_rows, d, n), _vector(where, "dst_rows", dst_rows, d, n), n,
        _vector(where, "seqlens", seqlens, d, rows), workspace.data_ptr(), workspace.nbytes, _call_stream(stream, d))
    if st:
        _check(st, where)


def nf_kv_compact(layers: KVLayers, refs, block_table, workspace, stream=None):
    """Move the blocks in use to the front of the pool, in every layer, and
    renumber the table (see nf.h)."""
    where = "nf_kv_compact"
    d = _pool_args(where, layers, refs, block_table, workspace)
    rows, width = block_table.shape
    st = (_lib or load_library()).nf_kv_compact(layers.c, len(layers), refs.data_ptr(), block_table.data_ptr(), rows, width,
                                      workspace.data_ptr(), workspace.nbytes, _call_stream(stream, d))
    if st:
        _check(st, where)
