"""GB300 (sm_103a) modulation-fused NVFP4 activation producer and block-scaled GEMM.

Python binding of the C-ABI library ``libh3fp4.so`` (see ``include/h3fp4.h``).
The ``h3fp4_*`` functions mirror the C entry points one to one and take raw
device pointers (ints); the short-named helpers below them take torch tensors,
allocate outputs with torch and pass pointers plus torch's current stream, or
the one given as ``stream``; what they allocate belongs to that stream, as if
made under ``torch.cuda.stream(stream)``.  As with torch's own operators, the
order of the streams and the life of the tensors given are the caller's
(``Tensor.record_stream`` where one is dropped while that stream may use it).
Every arithmetic step runs in the library's CUDA kernels: there is no CPU or
PyTorch fallback, and every call raises if the library is missing or returns
an error status.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import struct
import typing

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libh3fp4.so")
MAX_SEGMENTS = 16

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_STATUS = ctypes.c_int

# (name, argtypes, restype) of every exported entry point.
_SIGNATURES = {
    "h3fp4_modulate_absmax": ([_P, _I64, _I64, _I64, _P, _P, _I64, _P, _I32, _P, _P, _P], _STATUS),
    "h3fp4_modulate_pack": ([_P, _I64, _I64, _I64, _I64, _P, _P, _I64, _P, _I32, _P, _P, _P, _P], _STATUS),
    "h3fp4_modulate_produce": ([_P, _I64, _I64, _I64, _I64, _P, _P, _I64, _P, _I32, _P, _P, _P, _P, _P], _STATUS),
    "h3fp4_swiglu_pack": ([_P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P], _STATUS),
    "h3fp4_quantize_pack": ([_P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P], _STATUS),
    "h3fp4_gemm_gated_residual": ([_P, _P, _P, _P, _P, _P, _P, _I64, _P, _I32, _P, _I64, _P, _I64, _I64, _I64, _I64,
                                   _I64, _P, _P], _STATUS),
    "h3fp4_gemm": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P], _STATUS),
    "h3fp4_swizzle_scales": ([_P, _I64, _I64, _I64, _P, _P], _STATUS),
    "h3fp4_swiglu_pack_noalloc": ([_P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P], _STATUS),
    "h3fp4_device_error": ([_P], _STATUS),
    "h3fp4_diag_producer_barrier_timeout": ([_P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, ctypes.c_uint32, _P],
                                            _STATUS),
    "h3fp4_diag_gemm_wait_timeout": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, ctypes.c_uint32, _P],
                                     _STATUS),
    "h3fp4_rope_axes": ([_P, _I64, _I64, _P, _I64, _I64, _I64, _I32, _I32, _P, _P], _STATUS),
    "h3fp4_kv_cache_write": ([_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _P, _P], _STATUS),
    "h3fp4_kv_cache_read": ([_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _P], _STATUS),
    "h3fp4_kv_attention": ([_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I32, _P, _P, _I32, ctypes.c_float, _I32, _I32,
                            _P, _I64, _P], _STATUS),
    "h3fp4_diag_attention_wait_timeout": ([_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I32, _P, _P, _I32, _P, _I64,
                                           ctypes.c_uint32, _P], _STATUS),
    "h3fp4_kv_attention_workspace": ([_I64, _I32, _I32, _I32, _I32, _I32, _I32], _I64),
    "h3fp4_norm_rope": ([_P, _P, _I64, _I32, ctypes.c_float, _P, _P], _STATUS),
    "h3fp4_norm_rope_backward": ([_P, _P, _I64, _I32, ctypes.c_float, _P, _P, _I64, _P], _STATUS),
    "h3fp4_norm_rope_backward_workspace": ([_I32], _I64),
    "h3fp4_kv_attention_sinks": ([_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I32, _P, _P, _I32, ctypes.c_float, _I32, _I32,
                                  _I32, _P, _I64, _P], _STATUS),
    "h3fp4_kv_attention_shared": ([_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I32, _P, _P, _I32, _P, _I32, ctypes.c_float,
                                   _I32, _P, _I64, _P], _STATUS),
    "h3fp4_kv_attention_shared_workspace": ([_I64, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32], _I64),
    "h3fp4_kv_tables": ([_P, _P], _STATUS),
    "h3fp4_status_string": ([_STATUS], ctypes.c_char_p),
    "h3fp4_build_info": ([], ctypes.c_char_p),
}

STATUS_NAMES = {0: "H3FP4_OK", 1: "H3FP4_ERR_NULL", 2: "H3FP4_ERR_ALIGN", 3: "H3FP4_ERR_SHAPE",
                4: "H3FP4_ERR_UNSUPPORTED", 5: "H3FP4_ERR_CUDA", 6: "H3FP4_ERR_DEVICE"}


class H3FP4Error(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func} failed: {STATUS_NAMES.get(status, status)} ({_status_text(status)})")


class GemmConfig(ctypes.Structure):
    _fields_ = [("n_group", _I32), ("stages", _I32), ("cta_pair", _I32), ("reserved", _I32)]


ROPE_MAX_AXES = 4
ROPE_LAYOUTS = {"interleaved": 0, "halves": 1}


# The header's structures in the platform's C layout.
_ROPE = struct.Struct("@PqPi4iii4x")
_KV_CACHE = struct.Struct("@PPPPiiii")
_KV_BATCH = struct.Struct("@PqPPii")
_NORM_HEADS = struct.Struct("@PqqPqqPii")
_NORM_GRADS = struct.Struct("@PqqPqqPqqPPii")
_KV_REQUESTS = struct.Struct("@PPPqPPPPPPPqiiiii4x")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _status_text(status: int) -> str:
    try:
        return lib().h3fp4_status_string(status).decode()
    except Exception:  # library not loadable: fall back to the enum name
        return STATUS_NAMES.get(status, "unknown")


def _call(name: str, *args) -> None:
    st = getattr(_lib or lib(), name)(*args)
    if st != 0:
        raise H3FP4Error(name, st)


def _too_large(func: str):
    """For 32-bit arguments whose `or` does not fit: ctypes drops high bits without a word.  (A negative one could hide a
    large one there, but negative ones are refused by the C entry in any case.)"""
    return H3FP4Error(func, 3)


def _offsets(seg_row_offsets):
    arr = (ctypes.c_int32 * len(seg_row_offsets))(*[int(v) for v in seg_row_offsets])
    return arr, len(seg_row_offsets) - 1


# ----------------------------------------------------------------------------
# Raw C-ABI mirrors: device pointers as ints, stream as an int handle (0 = default).
# ----------------------------------------------------------------------------
def h3fp4_modulate_absmax(x, ldx, m, d, shift, scale, ld_mod, seg_row_offsets, tensor_scale, scratch, stream=0):
    offs, nseg = _offsets(seg_row_offsets)
    _call("h3fp4_modulate_absmax", x, ldx, m, d, shift, scale, ld_mod, offs, nseg, tensor_scale, scratch, stream)


def h3fp4_modulate_pack(x, ldx, m, m_pad, d, shift, scale, ld_mod, seg_row_offsets, tensor_scale, qdata, sfa,
                        stream=0):
    offs, nseg = _offsets(seg_row_offsets)
    _call("h3fp4_modulate_pack", x, ldx, m, m_pad, d, shift, scale, ld_mod, offs, nseg, tensor_scale, qdata, sfa,
          stream)


def h3fp4_modulate_produce(x, ldx, m, m_pad, d, shift, scale, ld_mod, seg_row_offsets, tensor_scale, scratch, qdata,
                           sfa, stream=0):
    offs, nseg = _offsets(seg_row_offsets)
    _call("h3fp4_modulate_produce", x, ldx, m, m_pad, d, shift, scale, ld_mod, offs, nseg, tensor_scale, scratch,
          qdata, sfa, stream)


def h3fp4_swiglu_pack(gate, ldg, up, ldu, m, m_pad, f, tensor_scale, scratch, qdata, sfa, h_workspace=None,
                      stream=0):
    _call("h3fp4_swiglu_pack", gate, ldg, up, ldu, m, m_pad, f, tensor_scale, scratch, qdata, sfa, h_workspace,
          stream)


def h3fp4_quantize_pack(x, ldx, m, m_pad, d, tensor_scale, scratch, qdata, sfa, stream=0):
    _call("h3fp4_quantize_pack", x, ldx, m, m_pad, d, tensor_scale, scratch, qdata, sfa, stream)


def h3fp4_gemm(a_q, a_sf, a_ts, b_q, b_sf, b_ts, c, ldc, m, m_pad, n, k, cfg: GemmConfig | None = None, stream=0):
    _call("h3fp4_gemm", a_q, a_sf, a_ts, b_q, b_sf, b_ts, c, ldc, m, m_pad, n, k,
          ctypes.byref(cfg) if cfg is not None else None, stream)


def h3fp4_gemm_gated_residual(a_q, a_sf, a_ts, b_q, b_sf, b_ts, gate, ld_gate, seg_row_offsets, residual, ldr, out,
                              ldo, m, m_pad, n, k, cfg: GemmConfig | None = None, stream=0):
    offs, nseg = _offsets(seg_row_offsets)
    _call("h3fp4_gemm_gated_residual", a_q, a_sf, a_ts, b_q, b_sf, b_ts, gate, ld_gate, offs, nseg, residual, ldr,
          out, ldo, m, m_pad, n, k, ctypes.byref(cfg) if cfg is not None else None, stream)


def h3fp4_swizzle_scales(sf_logical, rows, cols, ld, sf_out, stream=0):
    _call("h3fp4_swizzle_scales", sf_logical, rows, cols, ld, sf_out, stream)


def h3fp4_swiglu_pack_noalloc(gate, ldg, up, ldu, m, m_pad, f, tensor_scale, qdata, sfa, stream=0):
    """The SwiGLU producer with library-owned static scratch, for callers that cannot allocate."""
    _call("h3fp4_swiglu_pack_noalloc", gate, ldg, up, ldu, m, m_pad, f, tensor_scale, qdata, sfa, stream)


NOALLOC_MAX_ELEMENTS = 1 << 22


def h3fp4_device_error() -> int:
    code = ctypes.c_uint32(0)
    _call("h3fp4_device_error", ctypes.byref(code))
    return code.value


def h3fp4_diag_producer_barrier_timeout(x, ldx, m, m_pad, d, tensor_scale, scratch, qdata, sfa, limit_us, stream=0):
    """Failure-detection check: the cooperative producer's grid barrier gives up after limit_us."""
    _call("h3fp4_diag_producer_barrier_timeout", x, ldx, m, m_pad, d, tensor_scale, scratch, qdata, sfa, limit_us,
          stream)


def h3fp4_diag_gemm_wait_timeout(a_q, a_sf, a_ts, b_q, b_sf, b_ts, c, ldc, m, m_pad, n, k, limit_us, stream=0):
    """Failure-detection check: the default GEMM with its loads withheld; its waits give up after limit_us."""
    _call("h3fp4_diag_gemm_wait_timeout", a_q, a_sf, a_ts, b_q, b_sf, b_ts, c, ldc, m, m_pad, n, k, limit_us, stream)


def h3fp4_rope_axes(x, x_token_stride, x_head_stride, out, out_token_stride, out_head_stride, tokens, heads, head_dim,
                    rope, stream=0):
    """`rope` (and `cache`, `batch` below): the structure's bytes, or None where the C entry takes NULL."""
    if not -1 <= (heads | head_dim) >> 31 <= 0:
        raise _too_large("h3fp4_rope_axes")
    _call("h3fp4_rope_axes", x, x_token_stride, x_head_stride, out, out_token_stride, out_head_stride, tokens, heads,
          head_dim, rope, stream)


def h3fp4_norm_rope(q, k, tokens, head_dim, eps, rope=None, stream=0):
    """`q` and `k` (of the gradients too): the structure's bytes, or None."""
    if not -1 <= head_dim >> 31 <= 0:
        raise _too_large("h3fp4_norm_rope")
    _call("h3fp4_norm_rope", q, k, tokens, head_dim, eps, rope, stream)


def h3fp4_norm_rope_backward(q, k, tokens, head_dim, eps, rope, workspace, workspace_bytes, stream=0):
    if not -1 <= head_dim >> 31 <= 0:
        raise _too_large("h3fp4_norm_rope_backward")
    _call("h3fp4_norm_rope_backward", q, k, tokens, head_dim, eps, rope, workspace, workspace_bytes, stream)


def h3fp4_norm_rope_backward_workspace(head_dim) -> int:
    n = lib().h3fp4_norm_rope_backward_workspace(head_dim) if -1 <= head_dim >> 31 <= 0 else -1
    if n < 0:
        raise H3FP4Error("h3fp4_norm_rope_backward_workspace", 3)
    return n


def h3fp4_kv_cache_write(cache, batch, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, tokens,
                         rope=None, stream=0):
    _call("h3fp4_kv_cache_write", cache, batch, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride,
          tokens, rope, stream)


def h3fp4_kv_cache_read(cache, batch, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, tokens,
                        stream=0):
    _call("h3fp4_kv_cache_read", cache, batch, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride,
          tokens, stream)


def h3fp4_kv_attention(q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse, tokens, heads,
                       cache, batch, max_kv, softmax_scale, causal, window, workspace, workspace_bytes, stream=0):
    if not -1 <= (heads | max_kv | causal | window) >> 31 <= 0:
        raise _too_large("h3fp4_kv_attention")
    _call("h3fp4_kv_attention", q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse, tokens,
          heads, cache, batch, max_kv, softmax_scale, causal, window, workspace, workspace_bytes, stream)


def h3fp4_kv_attention_sinks(q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse, tokens, heads,
                             cache, batch, max_kv, softmax_scale, causal, window, sinks, workspace, workspace_bytes, stream=0):
    if not -1 <= (heads | max_kv | causal | window | sinks) >> 31 <= 0:
        raise _too_large("h3fp4_kv_attention_sinks")
    _call("h3fp4_kv_attention_sinks", q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse, tokens,
          heads, cache, batch, max_kv, softmax_scale, causal, window, sinks, workspace, workspace_bytes, stream)


def h3fp4_kv_attention_shared(q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse, tokens, heads,
                              cache, prefix, max_prefix, batch, max_kv, softmax_scale, causal, workspace, workspace_bytes,
                              stream=0):
    if not -1 <= (heads | max_prefix | max_kv | causal) >> 31 <= 0:
        raise _too_large("h3fp4_kv_attention_shared")
    _call("h3fp4_kv_attention_shared", q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse, tokens,
          heads, cache, prefix, max_prefix, batch, max_kv, softmax_scale, causal, workspace, workspace_bytes, stream)


def h3fp4_kv_attention_shared_workspace(tokens, heads, kv_heads, head_dim, groups, max_group_tokens, max_prefix, batch,
                                        max_tokens, max_kv) -> int:
    sizes = (heads, kv_heads, head_dim, groups, max_group_tokens, max_prefix, batch, max_tokens, max_kv)
    if not all(-1 <= x >> 31 <= 0 for x in sizes):
        raise _too_large("h3fp4_kv_attention_shared_workspace")
    n = lib().h3fp4_kv_attention_shared_workspace(tokens, *sizes)
    if n < 0:
        raise H3FP4Error("h3fp4_kv_attention_shared_workspace", 3)
    return n


def h3fp4_kv_tables(requests, stream=0):
    """`requests`: the structure's bytes."""
    _call("h3fp4_kv_tables", requests, stream)


def h3fp4_diag_attention_wait_timeout(q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse, tokens,
                                      heads, cache, batch, max_kv, workspace, workspace_bytes, limit_us, stream=0):
    """Runs few-query attention with copies that never complete (failure detection, see h3fp4.h)."""
    _call("h3fp4_diag_attention_wait_timeout", q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse,
          tokens, heads, cache, batch, max_kv, workspace, workspace_bytes, limit_us, stream)


def h3fp4_kv_attention_workspace(tokens, heads, kv_heads, head_dim, batch, max_tokens, max_kv) -> int:
    if not -1 <= (heads | kv_heads | head_dim | batch | max_tokens | max_kv) >> 31 <= 0:
        raise _too_large("h3fp4_kv_attention_workspace")
    n = lib().h3fp4_kv_attention_workspace(tokens, heads, kv_heads, head_dim, batch, max_tokens, max_kv)
    if n < 0:
        raise H3FP4Error("h3fp4_kv_attention_workspace", 3)
    return n


def h3fp4_build_info() -> str:
    return lib().h3fp4_build_info().decode()


# ----------------------------------------------------------------------------
# torch-tensor helpers (allocation with torch, pointers + current stream to the C ABI)
# ----------------------------------------------------------------------------
def sf_rows(rows: int) -> int:
    """Rows of a scale buffer: rows rounded up to a multiple of 128."""
    return -(-rows // 128) * 128


def sf_bytes(rows: int, width: int) -> int:
    return sf_rows(rows) * (width // 16)


def _stream(stream):
    import torch
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _empty(stream, *shape, dtype, device):
    """Uninitialised memory that belongs to the stream the call's kernels run on (None: torch's current one).  torch's
    allocator hands a block out again in the order of its own stream: a block of another stream may still be in use
    there, or come into use again before these kernels have finished with it."""
    empty = (_types or _dtypes())["empty"]
    if stream is None:
        return empty(*shape, dtype=dtype, device=device)
    import torch
    with torch.cuda.stream(stream):
        return empty(*shape, dtype=dtype, device=device)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")


def modulate_absmax(x, shift, scale, seg_row_offsets, *, tensor_scale=None, scratch=None, stream=None):
    """Pass 1: returns the FP32 tensor scale (1-element device tensor)."""
    import torch
    _need_cuda(x, shift, scale)
    m, d = x.shape
    if tensor_scale is None:
        tensor_scale = _empty(stream, 1, dtype=torch.float32, device=x.device)
    if scratch is None:
        scratch = _empty(stream, 2, dtype=torch.int32, device=x.device)
    h3fp4_modulate_absmax(x.data_ptr(), x.stride(0), m, d, shift.data_ptr(), scale.data_ptr(), shift.stride(0),
                          seg_row_offsets, tensor_scale.data_ptr(), scratch.data_ptr(), _stream(stream))
    return tensor_scale


def modulate_pack(x, shift, scale, seg_row_offsets, tensor_scale, m_pad, *, qdata=None, sfa=None, stream=None):
    """Pass 2: returns (qdata [m_pad, d/2] uint8, sfa flat uint8 in the scale layout)."""
    import torch
    _need_cuda(x, shift, scale, tensor_scale)
    m, d = x.shape
    if qdata is None:
        qdata = _empty(stream, m_pad, d // 2, dtype=torch.uint8, device=x.device)
    if sfa is None:
        sfa = _empty(stream, sf_bytes(m_pad, d), dtype=torch.uint8, device=x.device)
    h3fp4_modulate_pack(x.data_ptr(), x.stride(0), m, m_pad, d, shift.data_ptr(), scale.data_ptr(), shift.stride(0),
                        seg_row_offsets, tensor_scale.data_ptr(), qdata.data_ptr(), sfa.data_ptr(), _stream(stream))
    return qdata, sfa


def modulate_produce(x, shift, scale, seg_row_offsets, m_pad, *, tensor_scale=None, scratch=None, qdata=None,
                     sfa=None, stream=None):
    """Both modulation-producer passes in one launch: returns (tensor_scale, qdata, sfa)."""
    import torch
    _need_cuda(x, shift, scale)
    m, d = x.shape
    dev = x.device
    if tensor_scale is None:
        tensor_scale = _empty(stream, 1, dtype=torch.float32, device=dev)
    if scratch is None:
        scratch = _empty(stream, 2, dtype=torch.int32, device=dev)
    if qdata is None:
        qdata = _empty(stream, m_pad, d // 2, dtype=torch.uint8, device=dev)
    if sfa is None:
        sfa = _empty(stream, sf_bytes(m_pad, d), dtype=torch.uint8, device=dev)
    h3fp4_modulate_produce(x.data_ptr(), x.stride(0), m, m_pad, d, shift.data_ptr(), scale.data_ptr(),
                           shift.stride(0), seg_row_offsets, tensor_scale.data_ptr(), scratch.data_ptr(),
                           qdata.data_ptr(), sfa.data_ptr(), _stream(stream))
    return tensor_scale, qdata, sfa


def swiglu_pack(gate, up, m_pad, *, h_workspace=None, tensor_scale=None, scratch=None, qdata=None, sfa=None,
                stream=None):
    """SwiGLU producer: returns (tensor_scale, qdata, sfa)."""
    import torch
    _need_cuda(gate, up, h_workspace)
    m, f = gate.shape
    dev = gate.device
    if tensor_scale is None:
        tensor_scale = _empty(stream, 1, dtype=torch.float32, device=dev)
    if scratch is None:
        scratch = _empty(stream, 2, dtype=torch.int32, device=dev)
    if qdata is None:
        qdata = _empty(stream, m_pad, f // 2, dtype=torch.uint8, device=dev)
    if sfa is None:
        sfa = _empty(stream, sf_bytes(m_pad, f), dtype=torch.uint8, device=dev)
    h3fp4_swiglu_pack(gate.data_ptr(), gate.stride(0), up.data_ptr(), up.stride(0), m, m_pad, f,
                      tensor_scale.data_ptr(), scratch.data_ptr(), qdata.data_ptr(), sfa.data_ptr(),
                      h_workspace.data_ptr() if h_workspace is not None else None, _stream(stream))
    return tensor_scale, qdata, sfa


def quantize_pack(x, m_pad, *, tensor_scale=None, scratch=None, qdata=None, sfa=None, stream=None):
    """NVFP4 producer of a plain bf16 activation (both passes): returns (tensor_scale, qdata, sfa)."""
    import torch
    _need_cuda(x)
    m, d = x.shape
    dev = x.device
    if tensor_scale is None:
        tensor_scale = _empty(stream, 1, dtype=torch.float32, device=dev)
    if scratch is None:
        scratch = _empty(stream, 2, dtype=torch.int32, device=dev)
    if qdata is None:
        qdata = _empty(stream, m_pad, d // 2, dtype=torch.uint8, device=dev)
    if sfa is None:
        sfa = _empty(stream, sf_bytes(m_pad, d), dtype=torch.uint8, device=dev)
    h3fp4_quantize_pack(x.data_ptr(), x.stride(0), m, m_pad, d, tensor_scale.data_ptr(), scratch.data_ptr(),
                        qdata.data_ptr(), sfa.data_ptr(), _stream(stream))
    return tensor_scale, qdata, sfa


def gemm(a_q, a_sf, a_ts, b_q, b_sf, b_ts, m, *, out=None, cfg: GemmConfig | None = None, stream=None):
    """C[m, n] bf16 (returned as int16 patterns unless `out` is given)."""
    import torch
    _need_cuda(a_q, a_sf, a_ts, b_q, b_sf, b_ts, out)
    m_pad, kh = a_q.shape
    n = b_q.shape[0]
    if out is None:
        out = _empty(stream, m, n, dtype=torch.int16, device=a_q.device)
    h3fp4_gemm(a_q.data_ptr(), a_sf.data_ptr(), a_ts.data_ptr(), b_q.data_ptr(), b_sf.data_ptr(), b_ts.data_ptr(),
               out.data_ptr(), out.stride(0), m, m_pad, n, 2 * kh, cfg, _stream(stream))
    return out


def gemm_gated_residual(a_q, a_sf, a_ts, b_q, b_sf, b_ts, m, gate, seg_row_offsets, residual, *, out=None,
                       cfg: GemmConfig | None = None, stream=None):
    """out = RN_bf16(residual + RN_bf16(gate_s * C)) with C the GEMM result; pass
    out=residual to update the residual in place.  Returns out (int16 bf16 patterns)."""
    import torch
    _need_cuda(a_q, a_sf, a_ts, b_q, b_sf, b_ts, gate, residual, out)
    m_pad, kh = a_q.shape
    n = b_q.shape[0]
    if out is None:
        out = _empty(stream, m, n, dtype=torch.int16, device=a_q.device)
    h3fp4_gemm_gated_residual(a_q.data_ptr(), a_sf.data_ptr(), a_ts.data_ptr(), b_q.data_ptr(), b_sf.data_ptr(),
                              b_ts.data_ptr(), gate.data_ptr(), gate.stride(0), seg_row_offsets,
                              residual.data_ptr(), residual.stride(0), out.data_ptr(), out.stride(0), m, m_pad, n,
                              2 * kh, cfg, _stream(stream))
    return out


def swizzle_scales(sf_logical, *, out=None, stream=None):
    """Logical [rows, cols] uint8 scales -> flat scale-layout bytes (rows padded to 128)."""
    import torch
    _need_cuda(sf_logical, out)
    rows, cols = sf_logical.shape
    if out is None:
        out = _empty(stream, sf_rows(rows) * cols, dtype=torch.uint8, device=sf_logical.device)
    h3fp4_swizzle_scales(sf_logical.data_ptr(), rows, cols, sf_logical.stride(0), out.data_ptr(), _stream(stream))
    return out


# ----------------------------------------------------------------------------
# Rotary positions, the 8-bit key/value cache, and attention over it.  bf16
# tensors are torch.bfloat16 or int16 patterns; outputs take their input's type.
# The checks stand between a caller's tensors and raw pointers, so each call
# makes all of them; they are written to cost little (a decoding step's calls
# take longer on the host than on the GPU).
# ----------------------------------------------------------------------------
_types = None


def _dtypes():
    global _types
    if _types is None:
        import torch
        _types = {"bf16": (torch.bfloat16, torch.int16), "i32": torch.int32, "i64": torch.int64, "f32": torch.float32,
                  "f64": torch.float64, "u8": torch.uint8, "empty": torch.empty}
    return _types


def _need_array(t, name, dtype, ndim, device):
    """A contiguous array of this element type on the device; returns its address."""
    if not (t.get_device() == device >= 0 and t.dtype is _dtypes()[dtype] and t.dim() == ndim and t.is_contiguous()):
        _refuse(t, name, f"a contiguous {ndim}-D {_dtypes()[dtype]} tensor", device)
    return t.data_ptr()


def _need_tokens(t, name, shape=None, device=None):
    """A [tokens, heads, head_dim] array of bf16 values or patterns on the device (None: any); returns its address and
    strides."""
    s, at = t.stride(), t.get_device()
    if not (at >= 0 and (at == device or device is None) and t.dtype in _dtypes()["bf16"] and len(s) == 3 and (s[2] == 1 or t.shape[2] == 1)
            and (shape is None or t.shape == shape)):
        _refuse(t, name, f"a [tokens, heads, head_dim] tensor {'' if shape is None else tuple(shape)} of bf16 values "
                         "(bfloat16 or int16) with contiguous channels", -1 if device is None else device)
    return t.data_ptr(), s[0], s[1]


def _need_device(of, name, device):
    if of._device != device:
        raise ValueError(f"{name}: its tensors lie on CUDA device {of._device}, the call's on {device}")


def _refuse(t, name, what, device):
    raise ValueError(f"{name}: {what} on {'a CUDA device' if device < 0 else f'CUDA device {device}'} is wanted, got "
                     f"{tuple(t.shape)} {t.dtype} strides {t.stride()} on {t.device}")


def _raw_stream(stream, t):
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _fixed(*names):
    """Attributes that are set once, in __init__, under a leading underscore: the C structure is packed there too, and
    another tensor in their place would need another one."""
    return (property(operator.attrgetter("_" + n)) for n in names)


class Rope:
    """Rotary positions of a call's tokens: ``positions`` [tokens, axes] float32,
    ``freqs`` [sum(dims)/2] float64 in radians per unit of position (the pairs of
    axis 0 first), ``dims`` the channels each axis turns, ``layout`` how a pair lies
    in its axis' channels: "interleaved" (2j, 2j+1) or "halves" (j, j + dims/2)."""

    __slots__ = ("_positions", "_freqs", "_dims", "_layout", "_device", "_struct")
    positions, freqs, dims, layout, device = _fixed("positions", "freqs", "dims", "layout", "device")

    def __init__(self, positions, freqs, dims, layout="interleaved"):
        device, n = positions.get_device(), len(dims)
        p, f = _need_array(positions, "positions", "f32", 2, device), _need_array(freqs, "freqs", "f64", 1, device)
        if not 1 <= n <= ROPE_MAX_AXES or positions.shape[1] < n or 2 * freqs.shape[0] < sum(dims) or layout not in ROPE_LAYOUTS:
            raise ValueError(f"rope: dims {tuple(dims)}, layout {layout!r} (one of {sorted(ROPE_LAYOUTS)}) with positions "
                             f"{tuple(positions.shape)} and {freqs.shape[0]} frequencies")
        self._positions, self._freqs, self._dims, self._layout, self._device = positions, freqs, tuple(dims), layout, device
        self._struct = _ROPE.pack(p, positions.shape[1], f, n, *dims, *(0,) * (ROPE_MAX_AXES - n), ROPE_LAYOUTS[layout], 0)

    def struct(self, inverse=False) -> bytes:
        return self._struct[:-8] + struct.pack("@i4x", 1) if inverse else self._struct


def rope_frequencies(dims, theta=10000.0, device="cuda"):
    """theta^(-2j/d) for the pairs j of each axis' d channels: ``freqs`` of a Rope."""
    import torch
    return torch.cat([theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / max(d, 1)) for d in dims]).to(device)


def _positions_for(rope, tokens, device):
    _need_device(rope, "rope", device)
    if rope._positions.shape[0] < tokens:
        raise ValueError(f"rope: {rope._positions.shape[0]} positions for {tokens} tokens")


def rope_axes(x, rope: Rope, *, inverse=False, out=None, stream=None):
    """x [tokens, heads, head_dim] turned by its tokens' positions; inverse=True turns
    back (and is the gradient).  out=x works in place.  Returns out."""
    device, shape = x.get_device(), x.shape
    xs = _need_tokens(x, "x")
    _positions_for(rope, shape[0], device)
    if out is None:
        out = x.new_empty(shape) if stream is None else _empty(stream, shape, dtype=x.dtype, device=x.device)
    h3fp4_rope_axes(*xs, *_need_tokens(out, "out", shape, device), *shape, rope.struct(inverse), _raw_stream(stream, x))
    return out


def _norm_side(x, name, weight, shape, device):
    """A side's array, weight and what the structures say of the weight."""
    its = x.shape
    if len(its) != 3 or its[0] != shape[0] or its[2] != shape[2]:
        _refuse(x, name, f"a [{shape[0]}, heads, {shape[2]}] tensor", device)
    at = _need_tokens(x, name, None, device)
    if weight is None:
        return at, 0, 0
    wide = weight.dtype is _dtypes()["f32"]
    if not (weight.get_device() == device and weight.shape == shape[2:] and weight.is_contiguous()
            and (wide or weight.dtype in _dtypes()["bf16"])):
        _refuse(weight, f"{name}_weight", f"a contiguous [{shape[2]}] tensor of bf16 values or float32", device)
    return at, weight.data_ptr(), int(wide)


def _out_like(x, out, name, device, stream):
    """The output given for x, or a new contiguous one; its address and strides."""
    shape = x.shape
    if out is not None:
        return out, _need_tokens(out, name, shape, device)
    out = _empty(stream, shape, dtype=x.dtype, device=x.device)
    return out, (out.data_ptr(), shape[1] * shape[2], shape[2])


def norm_rope(q, k=None, *, q_weight=None, k_weight=None, rope: Rope | None = None, eps=1e-6, q_out=None, k_out=None,
              stream=None):
    """RMS norm over the channels of every head of q (and k) [tokens, heads, head_dim], times the side's weight
    [head_dim] (bf16 or float32; None: ones), then turned by ``rope`` (None: not), rounded once.  q and k may have
    different numbers of heads; q_out=q works in place.  Returns (q_out, k_out); k_out is None without k."""
    device, shape = q.get_device(), q.shape
    _need_tokens(q, "q")                   # (three dimensions and a device: what the rest goes by)
    at, w, wide = _norm_side(q, "q", q_weight, shape, device)
    q_out, to = _out_like(q, q_out, "q_out", device, stream)
    q_side, k_side = _NORM_HEADS.pack(*at, *to, w, shape[1], wide), None
    if k is not None:
        at, w, wide = _norm_side(k, "k", k_weight, shape, device)
        k_out, to = _out_like(k, k_out, "k_out", device, stream)
        k_side = _NORM_HEADS.pack(*at, *to, w, k.shape[1], wide)
    elif k_weight is not None or k_out is not None:
        raise ValueError("k: a weight or an output without k")
    rope_at = None
    if rope is not None:
        _positions_for(rope, shape[0], device)
        rope_at = rope._struct
    h3fp4_norm_rope(q_side, k_side, shape[0], shape[2], eps, rope_at, _raw_stream(stream, q))
    return q_out, k_out


def norm_rope_backward(q_grad, k_grad, q, k=None, *, q_weight=None, k_weight=None, rope: Rope | None = None, eps=1e-6,
                       q_out=None, k_out=None, q_weight_grad=None, k_weight_grad=None, workspace=None, stream=None):
    """Gradients of ``norm_rope`` from those of its outputs and its inputs (nothing else is kept of the forward pass).
    Returns (dq, dk, dq_weight, dk_weight): dq and dk like q and k (q_out=q_grad works in place), the weights' float32
    [head_dim], None where there is no weight."""
    device, shape = q.get_device(), q.shape
    _need_tokens(q, "q")
    q_side, q_out, q_weight_grad = _norm_grad_side(q_grad, q, "q", q_weight, q_out, q_weight_grad, shape, device, stream)
    k_side = None
    if k is not None:
        k_side, k_out, k_weight_grad = _norm_grad_side(k_grad, k, "k", k_weight, k_out, k_weight_grad, shape, device, stream)
    elif any(t is not None for t in (k_grad, k_weight, k_out, k_weight_grad)):
        raise ValueError("k: gradients, a weight or an output without k")
    rope_at = None
    if rope is not None:
        _positions_for(rope, shape[0], device)
        rope_at = rope._struct
    sums = q_weight_grad is not None or k_weight_grad is not None
    at, have, workspace = _workspace(workspace, _norm_workspace(device, shape[2]) if sums else 0, device, stream, q)
    h3fp4_norm_rope_backward(q_side, k_side, shape[0], shape[2], eps, rope_at, at, have, _raw_stream(stream, q))
    return q_out, k_out, q_weight_grad, k_weight_grad


def _norm_grad_side(g, x, name, weight, out, dw, shape, device, stream):
    """A side's structure, and its gradients."""
    at, w, wide = _norm_side(x, name, weight, shape, device)
    gt = _need_tokens(g, name + "_grad", x.shape, device)
    out, to = _out_like(x, out, name + "_out", device, stream)
    dw_at = 0
    if dw is not None:
        if weight is None:
            raise ValueError(f"{name}_weight_grad: there is no {name}_weight")
        dw_at = _need_array(dw, name + "_weight_grad", "f32", 1, device)
        if dw.shape != shape[2:]:
            _refuse(dw, name + "_weight_grad", f"a contiguous [{shape[2]}] tensor", device)
    elif weight is not None:
        dw = _empty(stream, shape[2:], dtype=_dtypes()["f32"], device=x.device)
        dw_at = dw.data_ptr()
    return _NORM_GRADS.pack(*gt, *at, *to, w, dw_at, x.shape[1], wide), out, dw


@functools.lru_cache(maxsize=64)           # a function of the head's channels and the device's SMs
def _norm_workspace(device, head_dim):
    return h3fp4_norm_rope_backward_workspace(head_dim)


class KVCache:
    """Keys and values in E4M3 pages: codes [num_pages, heads, page_size, head_dim]
    uint8 and scales [num_pages, heads] float32, for keys and values each."""

    __slots__ = ("_k_codes", "_k_scale", "_v_codes", "_v_scale", "_num_pages", "_heads", "_page_size", "_head_dim", "_device",
                 "_struct")
    k_codes, k_scale, v_codes, v_scale = _fixed("k_codes", "k_scale", "v_codes", "v_scale")
    num_pages, heads, page_size, head_dim, device = _fixed("num_pages", "heads", "page_size", "head_dim", "device")

    def __init__(self, k_codes, k_scale, v_codes, v_scale):
        device = k_codes.get_device()
        kc, vc = _need_array(k_codes, "k_codes", "u8", 4, device), _need_array(v_codes, "v_codes", "u8", 4, device)
        ks, vs = _need_array(k_scale, "k_scale", "f32", 2, device), _need_array(v_scale, "v_scale", "f32", 2, device)
        shape = k_codes.shape
        if v_codes.shape != shape or k_scale.shape != shape[:2] or v_scale.shape != shape[:2]:
            raise ValueError(f"cache: codes {tuple(shape)} and {tuple(v_codes.shape)} with scales {tuple(k_scale.shape)} and "
                             f"{tuple(v_scale.shape)}")
        self._k_codes, self._k_scale, self._v_codes, self._v_scale, self._device = k_codes, k_scale, v_codes, v_scale, device
        self._num_pages, self._heads, self._page_size, self._head_dim = shape
        self._struct = _KV_CACHE.pack(kc, vc, ks, vs, shape[0], shape[2], shape[1], shape[3])

    @classmethod
    def empty(cls, num_pages, page_size, heads, head_dim, device="cuda"):
        """A cache of uninitialised pages (a page's first write sets its scales)."""
        import torch
        codes = [torch.empty(num_pages, heads, page_size, head_dim, dtype=torch.uint8, device=device) for _ in "kv"]
        scale = [torch.ones(num_pages, heads, dtype=torch.float32, device=device) for _ in "kv"]
        return cls(codes[0], scale[0], codes[1], scale[1])

    def struct(self) -> bytes:
        return self._struct


def _kv_batch(page_table, length, cu_tokens, max_tokens, device) -> bytes:
    table, cu = _need_array(page_table, "page_table", "i32", 2, device), _need_array(cu_tokens, "cu_tokens", "i32", 1, device)
    batch, pages = page_table.shape
    n = 0
    if length is not None:
        n = _need_array(length, "lengths", "i32", 1, device)
    if cu_tokens.shape[0] != batch + 1 or (length is not None and length.shape[0] != batch):
        raise ValueError(f"page_table has {batch} sequences: cu_tokens of {batch + 1} and lengths of {batch} are wanted, got "
                         f"{cu_tokens.shape[0]} and {None if length is None else length.shape[0]}")
    return _KV_BATCH.pack(table, pages, n, cu, batch, max_tokens)


def kv_cache_write(cache: KVCache, k, v, page_table, held, cu_tokens, max_tokens, *, rope: Rope | None = None,
                   stream=None):
    """Quantises new keys and values [tokens, heads, head_dim] into the cache.  Sequence
    b's tokens are rows cu_tokens[b] .. cu_tokens[b+1]-1 and go to positions held[b] on
    (page_table [batch, pages], held [batch], cu_tokens [batch+1]: device int32);
    max_tokens is the most new tokens of any sequence.  With ``rope`` the keys are
    turned first.  The caller advances its lengths."""
    device, shape = cache._device, (k.shape[0], cache._heads, cache._head_dim)
    ks, vs = _need_tokens(k, "k", shape, device), _need_tokens(v, "v", shape, device)
    if held is None:
        raise ValueError("held: lengths before the call are wanted")
    if rope is not None:
        _positions_for(rope, shape[0], device)
    h3fp4_kv_cache_write(cache._struct, _kv_batch(page_table, held, cu_tokens, max_tokens, device), *ks, *vs, shape[0],
                         rope._struct if rope is not None else None, _raw_stream(stream, k))


def kv_cache_read(cache: KVCache, page_table, start, cu_tokens, tokens, max_tokens, *, k=None, v=None, stream=None):
    """The cache's keys and values as bf16: sequence b's positions start[b] on (start
    None: from 0), into rows cu_tokens[b] .. cu_tokens[b+1]-1 of [tokens, heads,
    head_dim] outputs.  Returns (k, v)."""
    import torch
    shape = (tokens, cache._heads, cache._head_dim)
    if k is None:
        k = _empty(stream, shape, dtype=torch.bfloat16, device=cache._k_codes.device)
    if v is None:
        v = _empty(stream, shape, dtype=torch.bfloat16, device=cache._k_codes.device)
    device = cache._device
    h3fp4_kv_cache_read(cache._struct, _kv_batch(page_table, start, cu_tokens, max_tokens, device),
                        *_need_tokens(k, "k", shape, device), *_need_tokens(v, "v", shape, device), tokens,
                        _raw_stream(stream, k))
    return k, v


@functools.lru_cache(maxsize=256)          # a function of the sizes and the device's SMs
def _attention_workspace(device, *sizes):
    return h3fp4_kv_attention_workspace(*sizes)


def kv_attention(q, cache: KVCache, page_table, kv_len, cu_tokens, max_tokens, max_kv, *, scale=None, causal=False,
                 window=0, sinks=0, out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of q [tokens, heads, head_dim] over the cache.  kv_len[b] counts all keys
    of sequence b, its new tokens' among them; query i of n stands at kv_len[b] - n + i and
    sees the keys before kv_len[b] that are not after it (causal) and not window or more
    before it (window > 0), unless they are among the first ``sinks``.  scale defaults to
    head_dim ** -0.5.  Returns (out, lse); lse [tokens, heads] float32 is None unless asked
    for."""
    device, shape, qs, out, to, lse, lse_at = _attention_arrays(q, cache, kv_len, out, lse, return_lse, stream)
    tokens, heads, dim = shape
    batch = _kv_batch(page_table, kv_len, cu_tokens, max_tokens, device)
    need = _attention_workspace(device, tokens, heads, cache._heads, dim, page_table.shape[0], max_tokens, max_kv)
    at, have, workspace = _workspace(workspace, need, device, stream, q)
    if sinks:
        h3fp4_kv_attention_sinks(*qs, *to, lse_at, tokens, heads, cache._struct, batch,
                                 max_kv, dim ** -0.5 if scale is None else scale, causal, window, sinks, at, have,
                                 _raw_stream(stream, q))
    else:
        h3fp4_kv_attention(*qs, *to, lse_at, tokens, heads, cache._struct, batch, max_kv,
                           dim ** -0.5 if scale is None else scale, causal, window, at, have, _raw_stream(stream, q))
    return out, lse


def _attention_arrays(q, cache, kv_len, out, lse, return_lse, stream):
    """Checks of what every attention call takes, and its outputs."""
    device, shape = q.get_device(), q.shape
    qs = _need_tokens(q, "q")
    _need_device(cache, "cache", device)
    tokens, heads, dim = shape
    if dim != cache._head_dim or heads % cache._heads or kv_len is None:
        raise ValueError(f"q: {heads} heads of {dim} for a cache of {cache.heads} heads of {cache.head_dim}"
                         if kv_len is not None else "kv_len: lengths are wanted")
    out, to = _out_like(q, out, "out", device, stream)
    lse_at = None
    if lse is None:
        if return_lse:
            lse = _empty(stream, (tokens, heads), dtype=_dtypes()["f32"], device=q.device)
            lse_at = lse.data_ptr()
    else:
        lse_at = _need_array(lse, "lse", "f32", 2, device)
        if lse.shape != (tokens, heads):
            _refuse(lse, "lse", f"a contiguous {(tokens, heads)} tensor", device)
    return device, shape, qs, out, to, lse, lse_at


def _workspace(workspace, need, device, stream, like):
    """Address and bytes of the caller's workspace, or of one made for the call (which the third result keeps)."""
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():   # (its bytes are written as they lie)
            _refuse(workspace, "workspace", "a contiguous tensor", device)
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if not need:
        return 0, 0, None
    workspace = _empty(stream, need, dtype=_dtypes()["u8"], device=like.device)
    return workspace.data_ptr(), need, workspace


class SharedPrefix:
    """Prefixes that groups of a call's sequences share: keys 0 .. kv_len[g] - 1 of row g of ``page_table``, seen by every
    query of rows cu_tokens[g] .. cu_tokens[g+1] - 1 (device int32, as for ``kv_attention``); max_tokens is the most rows
    of a group, max_kv the longest prefix."""

    __slots__ = ("_page_table", "_kv_len", "_cu_tokens", "_max_tokens", "_max_kv", "_device", "_struct")
    page_table, kv_len, cu_tokens = _fixed("page_table", "kv_len", "cu_tokens")
    max_tokens, max_kv, device = _fixed("max_tokens", "max_kv", "device")

    def __init__(self, page_table, kv_len, cu_tokens, max_tokens, max_kv):
        device = page_table.get_device()
        if kv_len is None:
            raise ValueError("kv_len: lengths are wanted")
        if not -1 <= (max_tokens | max_kv) >> 31 <= 0:
            raise _too_large("h3fp4_kv_attention_shared")
        self._struct = _kv_batch(page_table, kv_len, cu_tokens, max_tokens, device)
        self._page_table, self._kv_len, self._cu_tokens, self._device = page_table, kv_len, cu_tokens, device
        self._max_tokens, self._max_kv = max_tokens, max_kv


@functools.lru_cache(maxsize=256)          # a function of the sizes and the device's SMs
def _shared_workspace(device, *sizes):
    return h3fp4_kv_attention_shared_workspace(*sizes)


def kv_attention_shared(q, cache: KVCache, prefix: SharedPrefix, page_table, kv_len, cu_tokens, max_tokens, max_kv, *,
                        scale=None, causal=False, out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """``kv_attention`` of sequences that share prefixes: each query sees all of its group's prefix, and of its sequence's
    own keys what it sees in ``kv_attention``, under one softmax.  page_table and kv_len are those of the own keys alone,
    which begin on pages of their own.  The prefixes' pages are read once for a group, not once for a sequence.  Returns
    (out, lse)."""
    device, shape, qs, out, to, lse, lse_at = _attention_arrays(q, cache, kv_len, out, lse, return_lse, stream)
    _need_device(prefix, "prefix", device)
    tokens, heads, dim = shape
    batch = _kv_batch(page_table, kv_len, cu_tokens, max_tokens, device)
    need = _shared_workspace(device, tokens, heads, cache._heads, dim, prefix._page_table.shape[0], prefix._max_tokens,
                             prefix._max_kv, page_table.shape[0], max_tokens, max_kv)
    at, have, workspace = _workspace(workspace, need, device, stream, q)
    h3fp4_kv_attention_shared(*qs, *to, lse_at, tokens, heads, cache._struct, prefix._struct,
                              prefix._max_kv, batch, max_kv, dim ** -0.5 if scale is None else scale, causal, at, have,
                              _raw_stream(stream, q))
    return out, lse


class KVTables(typing.NamedTuple):
    """What ``kv_tables`` makes of a batch's lengths."""
    cu_tokens: object      # int32 [batch + 1]
    kv_len: object         # int32 [batch]
    slots: object          # int64 [tokens]
    positions: object      # float32 [tokens]
    free_at: object        # int32 [1]


def kv_tables(held, count, page_table, free_pages, free_at, page_size, num_pages, tokens, max_tokens, *, cu_tokens=None,
              kv_len=None, slots=None, positions=None, free_at_out=None, stream=None) -> KVTables:
    """The tables of a batch whose sequence b holds held[b] tokens and gets count[b] new ones (device int32 [batch], as are
    all lengths here): cu_tokens and kv_len for the cache and attention calls, pages for the new tokens, taken from
    free_pages[free_at[0]:] in the order of the sequences and written into page_table [batch, pages] where it has none
    yet, and of each new token its slot (page * page_size + its place in the page, int64) and its position (float32, as a
    Rope of one axis takes it).  slots and positions have ``tokens`` rows, of which those past the last token hold -1.
    The returned free_at counts what has been taken; the one given stays as it was."""
    device, batch, room, free = held.get_device(), *page_table.shape, free_pages.shape[0]
    at = (_need_array(held, "held", "i32", 1, device), _need_array(count, "count", "i32", 1, device),
          _need_array(page_table, "page_table", "i32", 2, device), room, _need_array(free_pages, "free_pages", "i32", 1, device),
          _need_array(free_at, "free_at", "i32", 1, device))
    if held.shape[0] != batch or count.shape[0] != batch or free_at.shape[0] != 1:
        raise ValueError(f"page_table has {batch} sequences: held and count of {batch} and one free_at are wanted, got "
                         f"{held.shape[0]}, {count.shape[0]} and {free_at.shape[0]}")
    if not 0 <= tokens < 1 << 31 or not -1 <= (page_size | num_pages | max_tokens | batch | free) >> 31 <= 0:
        raise _too_large("h3fp4_kv_tables")

    def out(t, name, kind, n):
        if t is None:
            t = _empty(stream, n, dtype=_dtypes()[kind], device=held.device)
            return t, t.data_ptr()
        to = _need_array(t, name, kind, 1, device)
        if t.shape[0] != n:
            _refuse(t, name, f"a contiguous [{n}] tensor", device)
        return t, to

    cu_tokens, cu_at = out(cu_tokens, "cu_tokens", "i32", batch + 1)
    kv_len, len_at = out(kv_len, "kv_len", "i32", batch)
    slots, slots_at = out(slots, "slots", "i64", tokens)
    positions, positions_at = out(positions, "positions", "f32", tokens)
    if not tokens:
        slots_at = positions_at = 16    # no rows have no address, but are not unwanted: tokens without a row are reported
    free_at_out, next_at = out(free_at_out, "free_at_out", "i32", 1)
    h3fp4_kv_tables(_KV_REQUESTS.pack(*at, next_at, cu_at, len_at, slots_at, positions_at, tokens, batch, max_tokens, free, num_pages,
                                      page_size), _raw_stream(stream, held))
    return KVTables(cu_tokens, kv_len, slots, positions, free_at_out)
