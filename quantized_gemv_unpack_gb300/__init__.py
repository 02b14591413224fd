"""Python binding of libqmv (fused dequantize-and-matvec for compressed-LLM decode on GB300).

Argument marshalling only: every function forwards to the C ABI of
``include/qmv.h`` under the same name. Device buffers are torch CUDA tensors
(or raw integer addresses); streams default to torch's current stream. A
failing call raises ``QmvError`` with the library's message. There is no
fallback: if ``libqmv.so`` has not been built, importing a call raises.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqmv.so")

QMV_ABI_VERSION = 1
QMV_GROUP = 128
QMV_MAX_SECTIONS = 8
QMV_MAX_M = 16
QMV_MAX_BATCH = 448

QMV_OK, QMV_ERR_ARG, QMV_ERR_ALIGN, QMV_ERR_UNSUPPORTED = 0, -1, -2, -3
QMV_ERR_CORRUPT, QMV_ERR_CUDA, QMV_ERR_TIMEOUT = -4, -5, -6
QMV_TERNARY2, QMV_INT4, QMV_CASS, QMV_CASS_MX, QMV_TERNARY2_SPARSE, QMV_TERNARY2_LUT, QMV_INT4_LUT = 1, 2, 3, 4, 5, 6, 7
QMV_FLAG_PATH_FMA, QMV_FLAG_PATH_MMA = 1, 2   # qmv_desc.flags: force the fp16-FMA or the tensor-core matvec kernel
QMV_FLAG_TEST_WAIT_TIMEOUT = 0x100           # qmv_desc.flags, testing only: the matvec's first wait gives up
QMV_KV_PAGE, QMV_KV_MAX_REQUESTS = 64, 8192  # tokens of a cache page; requests of a step
QMV_ROPE_MAX_PAIRS, QMV_ROPE_MAX_AXES = 128, 4
QMV_KV_INT8, QMV_KV_E4M3 = 1, 2              # code types of the KV cache
QMV_F32, QMV_BF16, QMV_F16 = 1, 2, 3         # activation types of the rope_* and kv8_* calls

# the exported C symbols (one per declaration in include/qmv.h)
EXPORTS = ("qmv_pack_desc", "qmv_pack_ternary", "qmv_pack_int4", "qmv_unpack", "qmv_run_ternary",
           "qmv_run_int4", "qmv_run_batch", "qmv_sparse_pack_host", "cass_pack_host", "cass_mx_pack_host", "cass_kv_encode", "cass_decode_draft", "cass_reconstruct",
           "cass_speculate_step", "moe_workspace_size", "moe_qmv_run", "moe_qmv_run_static",
           "kv8_desc", "kv_max_runs", "kv_plan", "rope_desc", "rope_run", "kv8_append", "kv8_read",
           "kv8_attend_workspace_size", "kv8_attend_init", "kv8_attend",
           "qmv_file_write", "qmv_file_open", "qmv_file_count", "qmv_file_tensor", "qmv_file_find", "qmv_file_load",
           "qmv_file_read_host", "qmv_file_close", "qmv_crc32", "qmv_check_status", "qmv_last_error")


class QmvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"qmv status {status}: {message}")
        self.status = status


class qmv_desc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("format", ctypes.c_uint32),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("group", ctypes.c_int32), ("n_symbols", ctypes.c_int32),
                ("off", ctypes.c_int64 * QMV_MAX_SECTIONS), ("bytes", ctypes.c_int64 * QMV_MAX_SECTIONS),
                ("total_bytes", ctypes.c_int64), ("flags", ctypes.c_uint64)]

    def sections(self):
        return [(int(self.off[i]), int(self.bytes[i])) for i in range(QMV_MAX_SECTIONS)]


class qmv_task(ctypes.Structure):
    _fields_ = [("desc", ctypes.POINTER(qmv_desc)), ("w", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class qmv_kv_desc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("type", ctypes.c_uint32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("off", ctypes.c_int64 * 2),
                ("bytes", ctypes.c_int64 * 2), ("total_bytes", ctypes.c_int64)]


class qmv_rope(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("axis", ctypes.c_uint8 * QMV_ROPE_MAX_PAIRS), ("turn", ctypes.c_uint64 * QMV_ROPE_MAX_PAIRS)]


class kv_plan_args(ctypes.Structure):
    _fields_ = [("n_requests", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("ld_table", ctypes.c_int64), ("max_runs", ctypes.c_int32)] + [
                    (n, ctypes.c_void_p) for n in ("lens", "add", "table", "ring", "ring_state", "ring_state_out", "lens_out",
                                                   "ctx", "status", "q_start", "slots", "positions", "runs", "held", "held_out")]


class kv8_append_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "q", "q_out")] + [
        (n, ctypes.c_int64) for n in ("ldk", "ldv", "ldq", "ldqo")] + [
        (n, ctypes.c_int32) for n in ("x_type", "q_out_type", "n_tokens", "n_q_heads", "n_runs")] + [
        (n, ctypes.c_void_p) for n in ("slots", "runs", "positions")] + [("ldp", ctypes.c_int64)]


class kv8_attend_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "out", "lse")] + [("ldq", ctypes.c_int64), ("ldo", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("x_type", "out_type", "n_requests", "n_tokens", "n_q_heads", "max_new")] + [
        (n, ctypes.c_void_p) for n in ("q_start", "ctx", "table")] + [
        ("ld_table", ctypes.c_int64), ("max_pages", ctypes.c_int32), ("window", ctypes.c_int32),
        ("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int
_DESC = ctypes.POINTER(qmv_desc)
_SIGS = {
    "qmv_pack_desc": (_I32, [_I32, _I64, _I64, ctypes.c_int32, _DESC]),
    "qmv_pack_ternary": (_I32, [_DESC, _P, _P, _P]),
    "qmv_pack_int4": (_I32, [_DESC, _P, _P, _P]),
    "qmv_unpack": (_I32, [_DESC, _P, _P, _P, _P]),
    "qmv_run_ternary": (_I32, [_DESC, _P, _P, _I32, _I64, _P, _I64, _P]),
    "qmv_run_int4": (_I32, [_DESC, _P, _P, _I32, _I64, _P, _I64, _P]),
    "qmv_run_batch": (_I32, [_I32, ctypes.POINTER(qmv_task), _I32, _I32, _P]),
    "cass_pack_host": (_I32, [_P, _I64, _I64, _P, _I64, _DESC, _P, _I64]),
    "cass_mx_pack_host": (_I32, [_P, _I64, _I64, _P, _I64, _DESC, _P, _I64]),
    "qmv_sparse_pack_host": (_I32, [_DESC, _P, _DESC, _P, _I64]),
    "cass_kv_encode": (_I32, [_P, _I64, _I64, _I64, _P, _I64, _DESC, _P, _I64, _P]),
    "cass_decode_draft": (_I32, [_DESC, _P, _P, _I32, _I64, _P, _I64, _P, _P]),
    "cass_reconstruct": (_I32, [_DESC, _P, _P, _I32, _I64, _P, _I64, _P, _P]),
    "cass_speculate_step": (_I32, [_DESC, _P, _P, _I32, _I64, _P, _P, _I64, _P]),
    "moe_workspace_size": (ctypes.c_size_t, [_I32, _I32, _I32, _I64, _I64]),
    "moe_qmv_run": (_I32, [_DESC, _DESC, _P, _I64, _I64, _I32, _P, _I32, _P, _I32, _I64, _P, _I64, _P,
                           ctypes.c_size_t, _P]),
    "moe_qmv_run_static": (_I32, [_DESC, _DESC, _P, _I64, _I64, _I32, _P, _I32, _P, _I32, _I64, _P, _I64, _P]),
    "kv8_desc": (_I32, [_I32, _I64, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(qmv_kv_desc)]),
    "kv_max_runs": (_I64, [_I64, _I64]),
    "kv_plan": (_I32, [ctypes.POINTER(kv_plan_args), _P]),
    "rope_desc": (_I32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                         ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(qmv_rope)]),
    "rope_run": (_I32, [ctypes.POINTER(qmv_rope), _P, _I32, _I64, ctypes.c_int32, _I64, _P, _I64, _P, _I32, _I64, _I32, _P]),
    "kv8_append": (_I32, [ctypes.POINTER(qmv_kv_desc), _P, ctypes.POINTER(qmv_rope), ctypes.POINTER(kv8_append_args), _P]),
    "kv8_read": (_I32, [ctypes.POINTER(qmv_kv_desc), _P, _P, _I64, _P, _P, _I32, _I64, _P]),
    "kv8_attend_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(qmv_kv_desc)]),
    "kv8_attend_init": (_I32, [ctypes.POINTER(qmv_kv_desc), _P, ctypes.c_size_t, _P]),
    "kv8_attend": (_I32, [ctypes.POINTER(qmv_kv_desc), _P, ctypes.POINTER(kv8_attend_args), _P]),
    "qmv_file_write": (_I32, [ctypes.c_char_p, _I32, ctypes.POINTER(ctypes.c_char_p), _DESC, ctypes.POINTER(_P)]),
    "qmv_file_open": (_I32, [ctypes.c_char_p, ctypes.POINTER(_P)]),
    "qmv_file_count": (_I32, [_P]),
    "qmv_file_tensor": (_I32, [_P, _I32, ctypes.c_char_p, _DESC]),
    "qmv_file_find": (_I32, [_P, ctypes.c_char_p]),
    "qmv_file_load": (_I32, [_P, _I32, _P, _I64, _P]),
    "qmv_file_read_host": (_I32, [_P, _I32, _P, _I64]),
    "qmv_file_close": (None, [_P]),
    "qmv_crc32": (ctypes.c_uint32, [_P, ctypes.c_size_t, ctypes.c_uint32]),
    "qmv_check_status": (_I32, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "qmv_last_error": (ctypes.c_char_p, []),
}


def lib():
    """The loaded libqmv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with quantized_gemv_unpack_gb300.build.build() "
                              "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def qmv_last_error() -> str:
    return lib().qmv_last_error().decode()


def _check(rc: int):
    if rc != QMV_OK:
        raise QmvError(rc, qmv_last_error())


def _ptr(t):
    """Device/host address of a torch tensor, a NumPy array, an int or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if hasattr(t, "ctypes"):
        return t.ctypes.data
    raise TypeError(f"cannot take the address of {type(t)}")


_raw_stream = None   # torch's current stream of a device as an integer, without making a Stream object


def _stream(stream):
    if stream is None:
        global _raw_stream
        import torch
        if _raw_stream is None:
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                lambda d: torch.cuda.current_stream(d).cuda_stream)
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ready(f, first, *rest):
    """Arguments of f as the C types it takes, so that a call that is made many times does not convert them each time."""
    return (first,) + tuple(t(v) for t, v in zip(f.argtypes[1:], rest))


def _rows(t):
    """(M, leading dimension) of a 2-D (or 1-D) activation/output tensor."""
    if t.dim() == 1:
        return 1, t.shape[0]
    return t.shape[0], t.stride(0)


# ----------------------------------------------------------------------------- layout and packing

def qmv_pack_desc(format: int, N: int, K: int, group: int = QMV_GROUP) -> qmv_desc:
    d = qmv_desc()
    _check(lib().qmv_pack_desc(format, N, K, group, ctypes.byref(d)))
    return d


def qmv_pack_ternary(desc: qmv_desc, w, packed, stream=None):
    _check(lib().qmv_pack_ternary(ctypes.byref(desc), _ptr(w), _ptr(packed), _stream(stream)))


def qmv_pack_int4(desc: qmv_desc, w, packed, stream=None):
    _check(lib().qmv_pack_int4(ctypes.byref(desc), _ptr(w), _ptr(packed), _stream(stream)))


def qmv_unpack(desc: qmv_desc, packed, q, scales=None, stream=None):
    _check(lib().qmv_unpack(ctypes.byref(desc), _ptr(packed), _ptr(q), _ptr(scales), _stream(stream)))


# ----------------------------------------------------------------------------- matvec

def qmv_run_ternary(desc: qmv_desc, w, x, y, stream=None):
    M, ldx = _rows(x)
    _, ldy = _rows(y)
    _check(lib().qmv_run_ternary(ctypes.byref(desc), _ptr(w), _ptr(x), M, ldx, _ptr(y), ldy, _stream(stream)))


def qmv_run_int4(desc: qmv_desc, w, x, y, stream=None):
    M, ldx = _rows(x)
    _, ldy = _rows(y)
    _check(lib().qmv_run_int4(ctypes.byref(desc), _ptr(w), _ptr(x), M, ldx, _ptr(y), ldy, _stream(stream)))


class Batch:
    """A prepared qmv_run_batch argument list. It keeps the descriptors, the ctypes
    arrays and the tensors (packed weights, x, y) alive for as long as it exists: the
    launch reads them through raw pointers, and memory that the caller's allocator took
    back and handed out again would otherwise be read as weights."""

    def __init__(self, format: int, tasks, M: int):
        self.format = format
        self.M = M
        self.descs = [t[0] for t in tasks]
        self.tensors = [tuple(t[1:]) for t in tasks]
        self.arr = (qmv_task * len(tasks))()
        for i, (d, w, x, y) in enumerate(tasks):
            _, ldx = _rows(x)
            _, ldy = _rows(y)
            self.arr[i] = qmv_task(ctypes.pointer(d), _ptr(w), _ptr(x), _ptr(y), ldx, ldy)

    def run(self, stream=None):
        _check(lib().qmv_run_batch(self.format, self.arr, len(self.arr), self.M, _stream(stream)))


def qmv_run_batch(format: int, tasks, M: int, stream=None):
    """tasks: list of (desc, w, x, y). Prefer ``Batch`` when the same list runs many times."""
    Batch(format, tasks, M).run(stream)


# ----------------------------------------------------------------------------- Cassandra

def _host_pack(fn, w_bf16_bits, calib_bf16_bits):
    import numpy as np
    w = np.ascontiguousarray(w_bf16_bits, dtype=np.uint16)
    c = np.ascontiguousarray(calib_bf16_bits, dtype=np.uint16)
    N, K = w.shape
    R = c.shape[0]
    d = qmv_desc()
    _check(fn(w.ctypes.data, N, K, c.ctypes.data, R, ctypes.byref(d), None, 0))
    out = np.zeros(d.total_bytes, dtype=np.uint8)
    _check(fn(w.ctypes.data, N, K, c.ctypes.data, R, ctypes.byref(d), out.ctypes.data, out.nbytes))
    return d, out


def cass_pack_host(w_bf16_bits, calib_bf16_bits):
    """Host packer: NumPy uint16 [N][K] weights and [R][K] calibration rows -> (desc, uint8 buffer)."""
    return _host_pack(lib().cass_pack_host, w_bf16_bits, calib_bf16_bits)


def qmv_sparse_pack_host(dense_desc: qmv_desc, dense_packed_host):
    """Flagged sparse ternary packer: a host copy (NumPy uint8) of a dense ternary buffer ->
    (desc, uint8 buffer) with all-zero 16 x 128 tiles left out."""
    import numpy as np
    src = np.ascontiguousarray(dense_packed_host, dtype=np.uint8)
    d = qmv_desc()
    _check(lib().qmv_sparse_pack_host(ctypes.byref(dense_desc), src.ctypes.data, ctypes.byref(d), None, 0))
    out = np.zeros(d.total_bytes, dtype=np.uint8)
    _check(lib().qmv_sparse_pack_host(ctypes.byref(dense_desc), src.ctypes.data, ctypes.byref(d), out.ctypes.data,
                                      out.nbytes))
    return d, out


def cass_kv_encode(kv, codebook, slot_words: int, packed=None, stream=None) -> qmv_desc:
    """Online KV encoder: kv device bf16 [T][ld] (one token per row), codebook NumPy uint8 [256]
    (the exponents in rank order). Returns the QMV_CASS descriptor; with packed (device uint8 of
    at least desc.total_bytes) also encodes into it. packed=None is a size query."""
    import numpy as np
    cb = np.ascontiguousarray(codebook, dtype=np.uint8)
    T, ld = _rows(kv)
    D = kv.shape[1]
    d = qmv_desc()
    _check(lib().cass_kv_encode(_ptr(kv), T, D, ld, cb.ctypes.data, slot_words, ctypes.byref(d),
                                _ptr(packed) if packed is not None else None,
                                packed.numel() if packed is not None else 0, _stream(stream)))
    return d


def cass_mx_pack_host(w_bf16_bits, calib_bf16_bits):
    """Cassandra-2 (MX) host packer, same arguments and result as cass_pack_host."""
    return _host_pack(lib().cass_mx_pack_host, w_bf16_bits, calib_bf16_bits)


def cass_decode_draft(desc: qmv_desc, packed, x, y=None, w_draft=None, stream=None):
    M, ldx = _rows(x)
    ldy = _rows(y)[1] if y is not None else 0
    _check(lib().cass_decode_draft(ctypes.byref(desc), _ptr(packed), _ptr(x), M, ldx, _ptr(y), ldy,
                                   _ptr(w_draft), _stream(stream)))


def cass_reconstruct(desc: qmv_desc, packed, x, y=None, w_out=None, stream=None):
    M, ldx = _rows(x)
    ldy = _rows(y)[1] if y is not None else 0
    _check(lib().cass_reconstruct(ctypes.byref(desc), _ptr(packed), _ptr(x), M, ldx, _ptr(y), ldy,
                                  _ptr(w_out), _stream(stream)))


def cass_speculate_step(desc: qmv_desc, packed, x, y_draft, y_target, stream=None):
    """x: bf16 [n_draft + 1][ldx] (row 0 the current token); y_draft [n_draft][ldy]; y_target
    [n_draft + 1][ldy] with the same ldy."""
    M, ldx = _rows(x)
    nd, ldy = _rows(y_draft)
    mt, ldy2 = _rows(y_target)
    if nd != M - 1 or mt != M or ldy2 != ldy:
        raise ValueError("x must have n_draft + 1 rows, y_draft n_draft and y_target n_draft + 1, one ldy")
    _check(lib().cass_speculate_step(ctypes.byref(desc), _ptr(packed), _ptr(x), nd, ldx, _ptr(y_draft),
                                     _ptr(y_target), ldy, _stream(stream)))


# ----------------------------------------------------------------------------- MoE

def moe_workspace_size(E: int, topk: int, M: int, H: int, I: int) -> int:
    return int(lib().moe_workspace_size(E, topk, M, H, I))


def moe_qmv_run(gateup_desc: qmv_desc, down_desc: qmv_desc, experts, expert_stride: int, down_off: int, E: int,
                logits, topk: int, x, y, workspace, stream=None):
    M, ldx = _rows(x)
    _, ldy = _rows(y)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().moe_qmv_run(ctypes.byref(gateup_desc), ctypes.byref(down_desc), _ptr(experts), expert_stride,
                             down_off, E, _ptr(logits), topk, _ptr(x), M, ldx, _ptr(y), ldy, _ptr(workspace),
                             ws_bytes, _stream(stream)))


QMV_MOE_STATIC_SCRATCH_BYTES = 2 * 1024 * 1024


def moe_qmv_run_static(gateup_desc: qmv_desc, down_desc: qmv_desc, experts, expert_stride: int, down_off: int,
                       E: int, logits, topk: int, x, y, stream=None):
    """moe_qmv_run without a caller workspace: for callers that cannot allocate device memory, the
    library's fixed device scratch array is used instead (see include/qmv.h)."""
    M, ldx = _rows(x)
    _, ldy = _rows(y)
    _check(lib().moe_qmv_run_static(ctypes.byref(gateup_desc), ctypes.byref(down_desc), _ptr(experts),
                                    expert_stride, down_off, E, _ptr(logits), topk, _ptr(x), M, ldx, _ptr(y), ldy,
                                    _stream(stream)))


# ----------------------------------------------------------------------------- paged 8-bit KV cache

# The calls of a serving step take many arguments that stay the same from step to step (buffers that a captured
# graph or a decode loop keeps), so each has a class that marshals them once, keeps its tensors alive like Batch,
# and issues the call with run(). Shapes, strides, types and devices are checked when it is made.

def _dtype(t):
    import torch
    code = {torch.float32: QMV_F32, torch.bfloat16: QMV_BF16, torch.float16: QMV_F16}.get(t.dtype)
    if code is None:
        raise TypeError(f"float32, bfloat16 or float16 expected, got {t.dtype}")
    return code


def _ints(name, t, shape, device):
    """An int32 tensor of the given shape (None: any extent), contiguous, on `device`."""
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous() or t.device != device:
        raise TypeError(f"{name}: a contiguous int32 tensor on {device} expected")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    return t


def _heads(name, t, heads, head_dim, device, tokens=None):
    """(address, token stride) of a [tokens][heads][head_dim] tensor whose heads lie side by side."""
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or t.shape[2] != head_dim:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected (tokens, {heads}, {head_dim})")
    if tokens is not None and t.shape[0] != tokens:
        raise ValueError(f"{name}: {t.shape[0]} tokens, expected {tokens}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != head_dim):
        raise ValueError(f"{name}: the heads of a token must lie side by side (strides {t.stride()})")
    row = t.shape[1] * head_dim
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else max(row, t.stride(0))


def _cache(desc, cache):
    import torch
    if cache.dtype != torch.uint8 or not cache.is_contiguous() or cache.numel() < desc.total_bytes:
        raise ValueError(f"cache: a contiguous uint8 tensor of at least {desc.total_bytes} bytes expected")
    return cache


def kv8_desc(type: int, n_pages: int, n_kv_heads: int, head_dim: int) -> qmv_kv_desc:
    """Layout of one layer's cache: allocate desc.total_bytes bytes (uint8) for it."""
    d = qmv_kv_desc()
    _check(lib().kv8_desc(type, n_pages, n_kv_heads, head_dim, ctypes.byref(d)))
    return d


def kv_max_runs(n_requests: int, n_tokens: int) -> int:
    return int(lib().kv_max_runs(n_requests, n_tokens))


class KvPlan:
    """kv_plan: block tables and slot maps of one step (see include/qmv.h). int32 device tensors lens, add [B],
    table [B][max_pages], ring [n_pages], ring_state [2] = (head, count); n_tokens is the number of new tokens' rows.
    run() fills slots, positions [n_tokens], runs [max_runs][2], q_start [B + 1], ctx, status [B], and lens_out and
    ring_state_out, which may be given as lens and ring_state to advance the state in place. A loop that takes tokens back
    (lens lowered between steps) gives held [B], the pages in each row of the table, too: held_out, which may be held, is
    then filled, and no page is lost."""

    def __init__(self, lens, add, table, ring, ring_state, n_tokens: int, lens_out=None, ring_state_out=None, held=None, held_out=None):
        import torch
        dev = lens.device
        B = lens.shape[0]
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
        self.lens, self.add = _ints("lens", lens, (B,), dev), _ints("add", add, (B,), dev)
        self.table, self.ring = _ints("table", table, (B, None), dev), _ints("ring", ring, (None,), dev)
        self.ring_state = _ints("ring_state", ring_state, (2,), dev)
        self.lens_out = new(B) if lens_out is None else _ints("lens_out", lens_out, (B,), dev)
        self.ring_state_out = new(2) if ring_state_out is None else _ints("ring_state_out", ring_state_out, (2,), dev)
        if held is None and held_out is not None:
            raise ValueError("held_out needs held")
        self.held = None if held is None else _ints("held", held, (B,), dev)
        self.held_out = None if held is None else new(B) if held_out is None else _ints("held_out", held_out, (B,), dev)
        max_runs = kv_max_runs(B, n_tokens)
        self.ctx, self.status, self.q_start = new(B), new(B), new(B + 1)
        self.slots, self.positions, self.runs = new(n_tokens), new(n_tokens), new(max_runs, 2)
        a = self.args = kv_plan_args(B, n_tokens, ring.shape[0], table.shape[1], table.shape[1], max_runs)
        for n in ("lens", "add", "table", "ring", "ring_state", "ring_state_out", "lens_out", "ctx", "status", "q_start",
                  "slots", "positions", "runs"):
            setattr(a, n, getattr(self, n).data_ptr())
        if held is not None:
            a.held, a.held_out = self.held.data_ptr(), self.held_out.data_ptr()
        self._call, self._args = lib().kv_plan, ctypes.byref(a)

    def run(self, stream=None):
        _check(self._call(self._args, _stream(stream)))


def rope_desc(head_dim: int, inv_freq, axis=None, interleaved: bool = False, n_axes: int | None = None) -> qmv_rope:
    """Rotation of the first 2 * len(inv_freq) values of each head; axis names the position axis of each pair
    (default: axis 0 for all)."""
    n = len(inv_freq)
    f = (ctypes.c_double * n)(*[float(x) for x in inv_freq])
    ax = None if axis is None else [int(x) for x in axis]
    if ax is not None and len(ax) != n:
        raise ValueError("axis and inv_freq differ in length")
    if n_axes is None:
        n_axes = max(ax) + 1 if ax else 1
    if n > QMV_ROPE_MAX_PAIRS:
        raise ValueError(f"{n} pairs, at most {QMV_ROPE_MAX_PAIRS}")
    r = qmv_rope()
    _check(lib().rope_desc(head_dim, 2 * n, n_axes, int(interleaved), f,
                           (ctypes.c_int32 * n)(*ax) if ax is not None else None, ctypes.byref(r)))
    return r


def _positions(rope, positions, tokens, device):
    p = positions if positions.dim() == 2 else positions.unsqueeze(0)
    if p.shape[0] < rope.n_axes or p.shape[1] < tokens:
        raise ValueError(f"positions: shape {tuple(positions.shape)}, expected at least ({rope.n_axes}, {tokens})")
    return _ints("positions", p, (None, None), device)


class Rope:
    """rope_run: x [tokens][heads][head_dim] rotated into out (same shape; may be x). positions: int32 [n_axes][tokens]
    (or [tokens] with one axis). inverse turns back, which is also the gradient."""

    def __init__(self, rope: qmv_rope, x, positions, out, inverse: bool = False):
        dev = x.device
        T, H = x.shape[0], x.shape[1]
        xp, ldx = _heads("x", x, None, rope.head_dim, dev)
        op, ldo = _heads("out", out, H, rope.head_dim, dev, T)
        pos = _positions(rope, positions, T, dev)
        self.keep = (rope, x, pos, out)
        self._call = lib().rope_run
        self._args = _ready(self._call, ctypes.byref(rope), xp, _dtype(x), T, H, ldx, pos.data_ptr(), pos.stride(0), op,
                            _dtype(out), ldo, int(inverse))

    def run(self, stream=None):
        _check(self._call(*self._args, _stream(stream)))


def rope_run(rope: qmv_rope, x, positions, out, inverse: bool = False, stream=None):
    """One call of Rope(...).run()."""
    Rope(rope, x, positions, out, inverse).run(stream)


class KvAppend:
    """kv8_append: write k, v [tokens][kv_heads][head_dim] to their slots (a KvPlan's slots and runs). With rope, k is
    rotated by positions first, and q [tokens][q_heads][head_dim], where given, is rotated into q_out."""

    def __init__(self, desc: qmv_kv_desc, cache, k, v, slots, runs, rope: qmv_rope | None = None, positions=None, q=None,
                 q_out=None):
        dev = cache.device
        H, D, T = desc.n_kv_heads, desc.head_dim, k.shape[0]
        a = self.args = kv8_append_args()
        a.k, a.ldk = _heads("k", k, H, D, dev)
        a.v, a.ldv = _heads("v", v, H, D, dev, T)
        a.x_type, a.n_tokens = _dtype(k), T
        if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
            raise TypeError("q, k and v must have one type")
        a.slots = _ints("slots", slots, (T,), dev).data_ptr()
        a.runs, a.n_runs = _ints("runs", runs, (None, 2), dev).data_ptr(), runs.shape[0]
        pos = None
        if rope is not None:
            if positions is None:
                raise ValueError("rope needs positions")
            pos = _positions(rope, positions, T, dev)
            a.positions, a.ldp = pos.data_ptr(), pos.stride(0)
        if q is not None:
            if q_out is None:
                raise ValueError("q needs q_out")
            a.q, a.ldq = _heads("q", q, None, D, dev, T)
            a.q_out, a.ldqo = _heads("q_out", q_out, q.shape[1], D, dev, T)
            a.q_out_type, a.n_q_heads = _dtype(q_out), q.shape[1]
        self.keep = (desc, _cache(desc, cache), k, v, slots, runs, rope, pos, q, q_out)
        self._call = lib().kv8_append
        self._args = (ctypes.byref(desc), cache.data_ptr(), ctypes.byref(rope) if rope is not None else None, ctypes.byref(a))

    def run(self, stream=None):
        _check(self._call(*self._args, _stream(stream)))


class KvRead:
    """kv8_read: the values that the codes of slots [n] stand for, into k_out and v_out [n][kv_heads][head_dim]."""

    def __init__(self, desc: qmv_kv_desc, cache, slots, k_out, v_out):
        dev = cache.device
        n = slots.shape[0]
        kp, ldk = _heads("k_out", k_out, desc.n_kv_heads, desc.head_dim, dev, n)
        vp, ldv = _heads("v_out", v_out, desc.n_kv_heads, desc.head_dim, dev, n)
        if ldk != ldv or k_out.dtype != v_out.dtype:
            raise ValueError("k_out and v_out must have one type and one stride")
        _ints("slots", slots, (n,), dev)
        self.keep = (desc, _cache(desc, cache), slots, k_out, v_out)
        self._call = lib().kv8_read
        self._args = _ready(self._call, ctypes.byref(desc), cache.data_ptr(), slots.data_ptr(), n, kp, vp, _dtype(k_out), ldk)

    def run(self, stream=None):
        _check(self._call(*self._args, _stream(stream)))


def kv8_workspace(desc: qmv_kv_desc, device):
    """A workspace for kv8_attend (uint8; 1 KB per SM and value of a head: 20 MB for heads of 128), ready for use on any
    stream: the call waits until it is cleared, unless it is made during a graph capture, to which it then belongs. Calls
    that overlap on the GPU need one each; layers that follow one another on a stream can share one."""
    import torch
    n = int(lib().kv8_attend_workspace_size(ctypes.byref(desc)))
    if n == 0:
        _check(QMV_ERR_ARG)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    with torch.cuda.device(ws.device):
        _check(lib().kv8_attend_init(ctypes.byref(desc), ws.data_ptr(), n, _stream(None)))
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
    return ws


class KvAttend:
    """kv8_attend: attention of q [tokens][q_heads][head_dim] over the cache into out (same shape), with a KvPlan's
    q_start [B + 1], ctx [B] and table [B][max_pages]. max_new bounds the new tokens of one request. slopes [q_heads]
    (fp32) and prefix [B] (int32) are device tensors; lse [tokens][q_heads] (fp32) is optional. Without a workspace
    one is made (kv8_workspace); layers of one stream should share it (its `workspace`). A step that mixes single tokens and
    a long prompt chunk is faster as two calls, over slices q_start[a:b + 1], ctx[a:b], table[a:b] with a max_new each."""

    def __init__(self, desc: qmv_kv_desc, cache, q, out, q_start, ctx, table, scale: float, max_new: int = 1,
                 softcap: float = 0.0, slopes=None, window: int = 0, prefix=None, lse=None, workspace=None):
        import torch
        dev = cache.device
        T, Hq, D = q.shape[0], q.shape[1], desc.head_dim
        B = ctx.shape[0]
        a = self.args = kv8_attend_args()
        a.q, a.ldq = _heads("q", q, None, D, dev)
        a.out, a.ldo = _heads("out", out, Hq, D, dev, T)
        a.x_type, a.out_type = _dtype(q), _dtype(out)
        a.n_requests, a.n_tokens, a.n_q_heads, a.max_new = B, T, Hq, max_new
        a.q_start = _ints("q_start", q_start, (B + 1,), dev).data_ptr()
        a.ctx = _ints("ctx", ctx, (B,), dev).data_ptr()
        a.table = _ints("table", table, (B, None), dev).data_ptr()
        a.ld_table, a.max_pages = table.shape[1], table.shape[1]
        a.window, a.scale, a.softcap = window, scale, softcap
        for name, t, shape in (("slopes", slopes, (Hq,)), ("lse", lse, (T, Hq))):
            if t is not None:
                if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous() or t.device != dev:
                    raise ValueError(f"{name}: a contiguous float32 tensor of shape {shape} on {dev} expected")
                setattr(a, name, t.data_ptr())
        if prefix is not None:
            a.prefix = _ints("prefix", prefix, (B,), dev).data_ptr()
        self.workspace = kv8_workspace(desc, dev) if workspace is None else workspace
        # a workspace made here: the streams that its memory is known to be used on
        self._streams = {_stream(None)} if workspace is None else None
        a.workspace, a.ws_bytes = self.workspace.data_ptr(), self.workspace.numel() * self.workspace.element_size()
        self.keep = (desc, _cache(desc, cache), q, out, q_start, ctx, table, slopes, prefix, lse)
        self._call = lib().kv8_attend
        self._args = (ctypes.byref(desc), cache.data_ptr(), ctypes.byref(a))

    def run(self, stream=None):
        s = _stream(stream)
        if self._streams is not None and s not in self._streams:
            self._use(s)
        _check(self._call(*self._args, s))

    def _use(self, s):
        """The caller does not see the workspace, so its memory is not given out again before stream s is done with it."""
        import torch
        if not torch.cuda.is_current_stream_capturing():   # a graph's memory lives as long as what it was captured from
            self.workspace.record_stream(torch.cuda.ExternalStream(s, device=self.workspace.device))
            self._streams.add(s)



# ----------------------------------------------------------------------------- packed-weight files

QMV_FILE_NAME_BYTES = 64


def qmv_crc32(data, crc: int = 0) -> int:
    """CRC-32 (zip polynomial) of a bytes-like object or a host NumPy array."""
    import numpy as np
    a = np.ascontiguousarray(np.frombuffer(data, dtype=np.uint8) if isinstance(data, (bytes, bytearray)) else data)
    return int(lib().qmv_crc32(_ptr(a), a.nbytes, crc))


def qmv_file_write(path: str, items):
    """items: [(name, qmv_desc, host buffer of desc.total_bytes bytes: NumPy array or CPU tensor)]."""
    n = len(items)
    names = (ctypes.c_char_p * n)(*[nm.encode() for nm, _, _ in items])
    descs = (qmv_desc * n)(*[d for _, d, _ in items])
    for _, d, b in items:
        nb = b.nbytes if hasattr(b, "nbytes") else b.numel() * b.element_size()
        if nb < d.total_bytes:
            raise ValueError("buffer smaller than desc.total_bytes")
        if hasattr(b, "is_cuda") and b.is_cuda:
            raise ValueError("qmv_file_write takes host buffers")
    bufs = (_P * n)(*[_ptr(b) for _, _, b in items])
    _check(lib().qmv_file_write(path.encode(), n, names, descs, bufs))


class QmvFile:
    """An open packed-weight file (qmv_file_open ... qmv_file_close)."""

    def __init__(self, path: str):
        h = _P()
        _check(lib().qmv_file_open(path.encode(), ctypes.byref(h)))
        self._h = h

    def __len__(self):
        return int(lib().qmv_file_count(self._h))

    def tensor(self, index: int):
        """(name, qmv_desc) of tensor `index`."""
        name = ctypes.create_string_buffer(QMV_FILE_NAME_BYTES)
        d = qmv_desc()
        _check(lib().qmv_file_tensor(self._h, index, name, ctypes.byref(d)))
        return name.value.decode(), d

    def find(self, name: str) -> int:
        i = lib().qmv_file_find(self._h, name.encode())
        if i < 0:
            _check(i)
        return int(i)

    def load(self, index: int, dst, stream=None):
        """Copy tensor `index` (CRC-checked) into the device buffer dst."""
        nb = dst.numel() * dst.element_size()
        _check(lib().qmv_file_load(self._h, index, _ptr(dst), nb, _stream(stream)))

    def read_host(self, index: int, dst):
        nb = dst.nbytes if hasattr(dst, "nbytes") else dst.numel() * dst.element_size()
        _check(lib().qmv_file_read_host(self._h, index, _ptr(dst), nb))

    def close(self):
        if self._h:
            lib().qmv_file_close(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


# ----------------------------------------------------------------------------- status

def qmv_check_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device error word; raises on CUDA failure."""
    code = ctypes.c_int32(0)
    rc = lib().qmv_check_status(_stream(stream), ctypes.byref(code))
    if rc == QMV_ERR_CUDA:
        _check(rc)
    return int(code.value)
