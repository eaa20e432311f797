"""ctypes binding of ``libbsa.so`` (declared in ``include/bsa.h``).

Argument marshalling only: every step of both forwards runs in the CUDA
library.  PyTorch is used for device memory and streams.  There is no CPU
fallback: if the library is missing or the device is not usable, the calls
raise.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

BSA_F32 = 0
BSA_BF16 = 1
BSA_TRA_SQRT_HALF_POWERS = 1  # tra_forward_ex flag: p = k + 1/2 as x^k sqrt(x)
BSA_TRA_BWD_DETERMINISTIC = 1  # tra_backward_ex flag: the two-kernel bf16 backward (no scratch, bit-repeatable)

_STATUS = {
    0: "BSA_OK",
    1: "BSA_ERR_NULLPTR",
    2: "BSA_ERR_SHAPE",
    3: "BSA_ERR_DTYPE",
    4: "BSA_ERR_UNSUPPORTED",
    5: "BSA_ERR_LAUNCH",
    6: "BSA_ERR_DEVICE",
    7: "BSA_ERR_ALIGN",
    8: "BSA_ERR_MEMORY",
    9: "BSA_ERR_SCRATCH_LIMIT",
}


class BsaError(RuntimeError):
    """A libbsa call returned a non-zero bsa_status, or the library is absent."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, "libbsa.so")


def load_library():
    """Load ``libbsa.so`` once and declare its C signatures."""
    global _LIB
    if _LIB is not None:
        return _LIB
    _LIB = open_library(library_path())
    return _LIB


@contextlib.contextmanager
def using_library(path):
    """Route every call of this module, inside the ``with`` block, to the
    library at ``path`` (e.g. the debug build, ``libbsa_debug.so``)."""
    global _LIB
    saved = load_library()
    _LIB = open_library(path)
    try:
        yield _LIB
    finally:
        _LIB = saved


def open_library(path):
    """Open a build of the library at ``path`` and declare its C signatures."""
    if not os.path.exists(path):
        raise BsaError(f"{path} is not built; run block_sparse_attention_tra_gb300.build.build()")
    lib = ctypes.CDLL(path)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.tra_forward.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, i32, vp]
    lib.tra_forward.restype = i32
    lib.tra_forward_ex.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, i32, i32, vp]
    lib.tra_forward_ex.restype = i32
    lib.tra_forward_host_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.tra_forward_host_workspace_size.restype = ctypes.c_size_t
    lib.tra_forward_host.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, i32, vp, ctypes.c_size_t, vp]
    lib.tra_forward_host.restype = i32
    lib.nsa_select_forward.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp]
    lib.nsa_select_forward.restype = i32
    lib.tra_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, i32, vp]
    lib.tra_backward.restype = i32
    lib.tra_backward_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, i32, i32, vp]
    lib.tra_backward_ex.restype = i32
    lib.tra_diff_forward.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, f32, i32, i32, vp]
    lib.tra_diff_forward.restype = i32
    lib.tra_diff_backward.argtypes = [vp] * 12 + [i32, i32, i32, i32, f32, f32, f32, i32, i32, vp]
    lib.tra_diff_backward.restype = i32
    lib.tra_diff_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, f32, i32, i32,
                                             vp]
    lib.tra_diff_forward_noalloc.restype = i32
    lib.nsa_select_fsa_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.nsa_select_fsa_workspace_size.restype = ctypes.c_size_t
    lib.nsa_select_forward_fsa.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp,
                                           ctypes.c_size_t, vp]
    lib.nsa_select_forward_fsa.restype = i32
    sz = ctypes.c_size_t
    lib.nsa_select_backward_workspace_size.argtypes = [i32] * 7
    lib.nsa_select_backward_workspace_size.restype = sz
    lib.nsa_select_backward.argtypes = [vp] * 10 + [i32] * 7 + [vp, sz, vp]
    lib.nsa_select_backward.restype = i32
    lib.nsa_cache_append.argtypes = [vp] * 12 + [i32] * 11 + [vp]
    lib.nsa_cache_append.restype = i32
    lib.nsa_select_decode_workspace_size.argtypes = [i32] * 7
    lib.nsa_select_decode_workspace_size.restype = sz
    lib.nsa_select_decode.argtypes = [vp] * 10 + [i32] * 8 + [vp, sz, vp]
    lib.nsa_select_decode.restype = i32
    lib.qk_norm_rope_forward.argtypes = [vp] * 9 + [i32] * 7 + [f32, f32, i32, i32, vp]
    lib.qk_norm_rope_forward.restype = i32
    lib.qk_norm_rope_backward_workspace_size.argtypes = [i32] * 5
    lib.qk_norm_rope_backward_workspace_size.restype = sz
    lib.qk_norm_rope_backward.argtypes = [vp] * 13 + [i32] * 7 + [f32, f32, i32, i32, vp, sz, vp]
    lib.qk_norm_rope_backward.restype = i32
    lib.nsa_cache4_append.argtypes = [vp] * 17 + [i32] * 10 + [f32, f32, i32, i32, vp]
    lib.nsa_cache4_append.restype = i32
    lib.nsa_cache4_read.argtypes = [vp] * 11 + [i32] * 8 + [vp]
    lib.nsa_cache4_read.restype = i32
    lib.nsa_cache4_decode_workspace_size.argtypes = [i32] * 7
    lib.nsa_cache4_decode_workspace_size.restype = sz
    lib.nsa_cache4_decode.argtypes = [vp] * 12 + [i32] * 8 + [vp, sz, vp]
    lib.nsa_cache4_decode.restype = i32
    lib.bsa_status_string.argtypes = [i32]
    lib.bsa_status_string.restype = ctypes.c_char_p
    lib.bsa_version.argtypes = []
    lib.bsa_version.restype = i32
    lib.bsa_device_error.argtypes = []
    lib.bsa_device_error.restype = i32
    lib.bsa_selftest_wait_timeout.argtypes = [ctypes.c_longlong, vp, vp]
    lib.bsa_selftest_wait_timeout.restype = i32
    lib.bsa_selftest_log2.argtypes = [vp, vp, vp, i32, vp]
    lib.bsa_selftest_log2.restype = i32
    lib.bsa_selftest_exp2.argtypes = [vp, vp, vp, i32, vp]
    lib.bsa_selftest_exp2.restype = i32
    lib.bsa_read_probe.argtypes = [vp, ctypes.c_size_t, i32, vp, vp]
    lib.bsa_read_probe.restype = i32
    return lib


def status_string(status: int) -> str:
    return load_library().bsa_status_string(int(status)).decode()


def device_error() -> int:
    """Read and clear the library's device error words (0 = none, 1 = a
    bounded wait inside a kernel timed out, -1 = could not be read)."""
    return int(load_library().bsa_device_error())


def _check(status: int, what: str):
    if status != 0:
        raise BsaError(f"{what} failed: {_STATUS.get(status, status)} ({status_string(status)})", status)


def tra_forward_raw(q, k, v, out, B, H, T, D, beta, p, dtype, stream=0) -> int:
    """Direct C call with integer device pointers; returns the bsa_status."""
    return load_library().tra_forward(q, k, v, out, B, H, T, D, float(beta), float(p), int(dtype), stream)


def tra_forward_ex_raw(q, k, v, out, B, H, T, D, beta, p, dtype, flags, stream=0) -> int:
    """Direct C call of tra_forward_ex with integer device pointers."""
    return load_library().tra_forward_ex(q, k, v, out, B, H, T, D, float(beta), float(p), int(dtype), int(flags),
                                         stream)


def tra_forward_host_workspace_size(B, H, T, D, dtype) -> int:
    """Device bytes tra_forward_host needs for its workspace (0 if the arguments are rejected)."""
    return int(load_library().tra_forward_host_workspace_size(B, H, T, D, int(dtype)))


def tra_forward_host_raw(q, k, v, out, B, H, T, D, beta, p, dtype, workspace, workspace_bytes, stream=0) -> int:
    """Direct C call of tra_forward_host: integer HOST pointers for q, k, v, out and a device workspace."""
    return load_library().tra_forward_host(q, k, v, out, B, H, T, D, float(beta), float(p), int(dtype), workspace,
                                           int(workspace_bytes), stream)


def tra_backward_raw(q, k, v, dout, dq, dk, dv, B, H, T, D, beta, p, dtype, stream=0) -> int:
    """Direct C call with integer device pointers; returns the bsa_status."""
    return load_library().tra_backward(q, k, v, dout, dq, dk, dv, B, H, T, D, float(beta), float(p), int(dtype),
                                       stream)


def tra_backward_ex_raw(q, k, v, dout, dq, dk, dv, B, H, T, D, beta, p, dtype, flags, stream=0) -> int:
    """Direct C call of tra_backward_ex with integer device pointers; returns the bsa_status."""
    return load_library().tra_backward_ex(q, k, v, dout, dq, dk, dv, B, H, T, D, float(beta), float(p), int(dtype),
                                          int(flags), stream)


def tra_diff_forward_raw(q1, q2, k1, k2, v, out, B, H, T, D, beta, lam, p, normalize, dtype, stream=0) -> int:
    """Direct C call with integer device pointers; returns the bsa_status."""
    return load_library().tra_diff_forward(q1, q2, k1, k2, v, out, B, H, T, D, float(beta), float(lam), float(p),
                                           int(bool(normalize)), int(dtype), stream)


def tra_diff_backward_raw(q1, q2, k1, k2, v, dout, dq1, dq2, dk1, dk2, dv, dlam, B, H, T, D, beta, lam, p,
                          normalize, dtype, stream=0) -> int:
    """Direct C call of tra_diff_backward with integer device pointers (dlam
    may be None); returns the bsa_status."""
    return load_library().tra_diff_backward(q1, q2, k1, k2, v, dout, dq1, dq2, dk1, dk2, dv, dlam, B, H, T, D,
                                            float(beta), float(lam), float(p), int(bool(normalize)), int(dtype),
                                            stream)


def tra_diff_forward_noalloc_raw(q1, q2, k1, k2, v, out, B, H, T, D, beta, lam, p, normalize, dtype,
                                 stream=0) -> int:
    """Direct call of the allocation-free differential entry point (for
    callers that cannot allocate device memory during the call: scratch lives
    in a fixed library-held device array); returns the bsa_status."""
    return load_library().tra_diff_forward_noalloc(q1, q2, k1, k2, v, out, B, H, T, D, float(beta), float(lam),
                                                   float(p), int(bool(normalize)), int(dtype), stream)


def nsa_select_forward_raw(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, block_size, S,
                           stream=0) -> int:
    """Direct C call with integer device pointers; returns the bsa_status."""
    return load_library().nsa_select_forward(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D,
                                             block_size, S, stream)


def nsa_select_fsa_workspace_size(B, Hq, Hkv, T, D, block_size, S) -> int:
    """Bytes of workspace ``nsa_select_forward_fsa`` needs (0 = sizes not accepted)."""
    return int(load_library().nsa_select_fsa_workspace_size(B, Hq, Hkv, T, D, block_size, S))


def nsa_select_forward_fsa_raw(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, block_size, S, workspace,
                               workspace_bytes, stream=0) -> int:
    """Direct C call with integer device pointers; returns the bsa_status."""
    return load_library().nsa_select_forward_fsa(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, block_size, S,
                                                 workspace, int(workspace_bytes), stream)


def nsa_select_backward_workspace_size(B, Hq, Hkv, T, D, block_size, S) -> int:
    """Bytes of workspace ``nsa_select_backward`` needs (0 = sizes not accepted)."""
    return int(load_library().nsa_select_backward_workspace_size(B, Hq, Hkv, T, D, block_size, S))


def nsa_select_backward_raw(q, k, v, block_idx, out, lse, dout, dq, dk, dv, B, Hq, Hkv, T, D, block_size, S,
                            workspace, workspace_bytes, stream=0) -> int:
    """Direct C call with integer device pointers; returns the bsa_status."""
    return load_library().nsa_select_backward(q, k, v, block_idx, out, lse, dout, dq, dk, dv, B, Hq, Hkv, T, D,
                                              block_size, S, workspace, int(workspace_bytes), stream)


def nsa_cache_append_raw(k, v, q, q_out, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens,
                         inv_freq, B, Hq, Hkv, n, D, page_size, max_pages, num_pages, rotary_dim, interleaved, dtype,
                         stream=0) -> int:
    """Direct C call with integer device pointers (q, q_out, new_lens and
    inv_freq may be None); returns the bsa_status."""
    return load_library().nsa_cache_append(k, v, q, q_out, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens,
                                           new_lens, inv_freq, B, Hq, Hkv, n, D, page_size, max_pages, num_pages,
                                           rotary_dim, int(bool(interleaved)), int(dtype), stream)


def nsa_select_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S) -> int:
    """Bytes of workspace ``nsa_select_decode`` needs (0 = sizes not accepted)."""
    return int(load_library().nsa_select_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S))


def nsa_select_decode_raw(q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx, out, lse, B, Hq,
                          Hkv, D, page_size, max_pages, num_pages, S, workspace, workspace_bytes, stream=0) -> int:
    """Direct C call with integer device pointers (block_idx and lse may be
    None); returns the bsa_status."""
    return load_library().nsa_select_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx,
                                            out, lse, B, Hq, Hkv, D, page_size, max_pages, num_pages, S, workspace,
                                            int(workspace_bytes), stream)


@functools.lru_cache(maxsize=256)
def _stride_array(numbers):
    return (ctypes.c_int64 * len(numbers))(*numbers)


def _strides(numbers):
    """Strides in elements as the C entry points take them (None: all contiguous); made once for each tuple."""
    return None if numbers is None else _stride_array(tuple(numbers))


def qk_norm_rope_forward_raw(q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq, strides, B, Hq, Hkv, T, D,
                             rotary_dim, interleaved, rotary_scale, eps, dtype, weight_dtype, stream=0) -> int:
    """Direct C call with integer device pointers (q_weight, k_weight,
    positions and inv_freq may be None); ``strides``: 12 numbers or None."""
    return load_library().qk_norm_rope_forward(q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq,
                                               _strides(strides), B, Hq, Hkv, T, D, rotary_dim, int(bool(interleaved)),
                                               float(rotary_scale), float(eps), int(dtype), int(weight_dtype), stream)


def qk_norm_rope_backward_workspace_size(B, Hq, Hkv, T, D) -> int:
    """Bytes of workspace ``qk_norm_rope_backward`` needs (0 = sizes not accepted)."""
    return int(load_library().qk_norm_rope_backward_workspace_size(B, Hq, Hkv, T, D))


def qk_norm_rope_backward_raw(q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, q_weight, k_weight, positions,
                              inv_freq, strides, B, Hq, Hkv, T, D, rotary_dim, interleaved, rotary_scale, eps, dtype,
                              weight_dtype, workspace, workspace_bytes, stream=0) -> int:
    """Direct C call with integer device pointers; ``strides``: 18 numbers or None."""
    return load_library().qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, q_weight, k_weight,
                                                positions, inv_freq, _strides(strides), B, Hq, Hkv, T, D, rotary_dim,
                                                int(bool(interleaved)), float(rotary_scale), float(eps), int(dtype),
                                                int(weight_dtype), workspace, int(workspace_bytes), stream)


def nsa_cache4_append_raw(k, v, q, q_out, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table,
                          cache_lens, new_lens, q_weight, k_weight, inv_freq, strides, B, Hq, Hkv, n, D, page_size,
                          max_pages, num_pages, rotary_dim, interleaved, rotary_scale, eps, dtype, weight_dtype,
                          stream=0) -> int:
    """Direct C call with integer device pointers (q, q_out, the factors,
    new_lens, the weights and inv_freq may be None); ``strides``: 9 numbers or
    None."""
    return load_library().nsa_cache4_append(k, v, q, q_out, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor,
                                            page_table, cache_lens, new_lens, q_weight, k_weight, inv_freq,
                                            _strides(strides), B, Hq, Hkv, n, D, page_size, max_pages, num_pages,
                                            rotary_dim, int(bool(interleaved)), float(rotary_scale), float(eps),
                                            int(dtype), int(weight_dtype), stream)


def nsa_cache4_read_raw(k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table, starts, cache_lens, k_out,
                        v_out, B, Hkv, n, D, page_size, max_pages, num_pages, dtype, stream=0) -> int:
    """Direct C call with integer device pointers (the factors and starts may
    be None); returns the bsa_status."""
    return load_library().nsa_cache4_read(k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table, starts,
                                          cache_lens, k_out, v_out, B, Hkv, n, D, page_size, max_pages, num_pages,
                                          int(dtype), stream)


def nsa_cache4_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S) -> int:
    """Bytes of workspace ``nsa_cache4_decode`` needs (0 = sizes not accepted)."""
    return int(load_library().nsa_cache4_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S))


def nsa_cache4_decode_raw(q, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table, cache_lens, block_idx,
                          out, lse, B, Hq, Hkv, D, page_size, max_pages, num_pages, S, workspace, workspace_bytes,
                          stream=0) -> int:
    """Direct C call with integer device pointers (the factors, block_idx and
    lse may be None); returns the bsa_status."""
    return load_library().nsa_cache4_decode(q, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table,
                                            cache_lens, block_idx, out, lse, B, Hq, Hkv, D, page_size, max_pages,
                                            num_pages, S, workspace, int(workspace_bytes), stream)


@contextlib.contextmanager
def _on_stream(torch, device, stream):
    """Within the block ``device`` is current and ``stream`` (None: the
    device's current one) is its current stream, so that allocations, copies
    and the library call all go there."""
    if stream is not None and not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream is not None and stream.device != device:
        raise BsaError(f"the stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _one_device(what, first, *others):
    """``first`` on a CUDA device and every other tensor (None: absent) on the same one; its index."""
    dev = first.get_device()
    if dev < 0:
        raise BsaError(f"{what} takes CUDA tensors (no CPU path)")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise BsaError(f"{what}: tensors on {first.device} and {t.device}")
    return dev


def _in_place(what, name, t, shape, *dtypes):
    """Tensors the library writes into (or reads in place) keep their memory: exact shape, type and layout."""
    if t.shape != shape:
        raise BsaError(f"{what}: {name} must be {list(shape)}, got {list(t.shape)}", 2)
    if t.dtype not in dtypes:
        raise BsaError(f"{what}: {name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}", 3)
    if not t.is_contiguous():
        raise BsaError(f"{what}: {name} must be contiguous", 2)


def _apart(what, name, result, own, *others):
    """Refuses a contiguous result whose memory meets another tensor's (None: absent), from that one's first element to
    its last; over ``own`` only where the two are the same elements (None: nowhere)."""
    begin = result.data_ptr()
    end = begin + result.numel() * result.element_size()
    if own is not None and not (own.data_ptr() == begin and own.is_contiguous()):
        others = (own, *others)
    for t in others:
        if t is not None:
            first = t.data_ptr()
            last = first + t.element_size() * sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
            if first < end and begin < last + t.element_size():
                raise BsaError(f"{what}: {name} overlaps another tensor of the call")


def _no_gradient(what, *tensors):
    """Refuses tensors that a gradient is asked of (called where autograd records): nothing would flow through the
    cache's codes, and what is written in place would change under a graph that holds it."""
    for t in tensors:
        if t is not None and t.requires_grad:
            raise BsaError(f"{what} has no gradient: call it under torch.no_grad() or on detached tensors")


def _int32(torch, t):
    return (t if t.dtype is torch.int32 else t.to(torch.int32)).contiguous()


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t):
    import torch

    if t.dtype == torch.float32:
        return BSA_F32
    if t.dtype == torch.bfloat16:
        return BSA_BF16
    raise BsaError(f"unsupported dtype {t.dtype}", 3)


def tra_forward(q, k, v, beta: float, p: float = 2.0, out=None, stream=None, sqrt_half_powers: bool = False):
    """Threshold rectified attention forward on CUDA tensors ``[B, H, T, D]``.

    ``out = ReLU(q k^T - tau(i))^p v`` with ``tau(i) = beta sqrt(2 ln(i+1)/D)``,
    causal, unnormalised; float32 or bfloat16 in, same dtype out.  Runs on
    ``stream`` (default: torch's current stream) without synchronising.
    ``sqrt_half_powers``: evaluate p = 0.5, 1.5, 2.5, 3.5 as x^k sqrt(x)
    (``tra_forward_ex`` with ``BSA_TRA_SQRT_HALF_POWERS``).
    """
    if q.device.type != "cuda":
        raise BsaError("tra_forward takes CUDA tensors (no CPU path)")
    if not (q.shape == k.shape == v.shape) or q.dim() != 4:
        raise BsaError("q, k, v must share one shape [B, H, T, D]", 2)
    if not (q.dtype == k.dtype == v.dtype):
        raise BsaError("q, k, v must share one dtype", 3)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if out is None:
        import torch

        out = torch.empty_like(q)
    B, H, T, D = q.shape
    if sqrt_half_powers:
        st = tra_forward_ex_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, T, D, beta, p,
                                _dtype_code(q), BSA_TRA_SQRT_HALF_POWERS, _stream_handle(stream))
    else:
        st = tra_forward_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, T, D,
                             beta, p, _dtype_code(q), _stream_handle(stream))
    _check(st, "tra_forward")
    return out


def tra_forward_host(q, k, v, beta: float, p: float = 2.0, out=None, workspace=None, stream=None):
    """Threshold rectified attention forward on CPU tensors ``[B, H, T, D]``
    (float32 or bfloat16; page-locked tensors, e.g. ``t.pin_memory()``, let the
    copies overlap the kernels).  The library streams chunks of heads through
    the GPU (``tra_forward_host``); ``workspace`` is a uint8 CUDA tensor of at
    least ``tra_forward_host_workspace_size`` bytes (allocated if None).  The
    call is asynchronous on ``stream`` (default: torch's current stream):
    keep q, k, v, out and the workspace alive, and synchronise ``stream``,
    before reading ``out`` or releasing them (the library's copies run on
    its own streams, which torch's allocators do not see)."""
    import torch

    if q.device.type != "cpu" or k.device.type != "cpu" or v.device.type != "cpu":
        raise BsaError("tra_forward_host takes host (CPU) tensors")
    if not (q.shape == k.shape == v.shape) or q.dim() != 4:
        raise BsaError("q, k, v must share one shape [B, H, T, D]", 2)
    if not (q.dtype == k.dtype == v.dtype):
        raise BsaError("q, k, v must share one dtype", 3)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if out.device.type != "cpu" or out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise BsaError("out must be a contiguous CPU tensor shaped and typed like q", 2)
    B, H, T, D = q.shape
    dt = _dtype_code(q)
    need = tra_forward_host_workspace_size(B, H, T, D, dt)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        if isinstance(stream, torch.cuda.Stream):
            workspace.record_stream(stream)  # not reused before `stream` passes this call
    st = tra_forward_host_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, T, D, beta, p, dt,
                              workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                              _stream_handle(stream))
    _check(st, "tra_forward_host")
    return out


_TRA_FUNCTION = None


def _tra_function():
    """The autograd function of the threshold attention (page
    "triton_threshold_attention.py", ThresholdRelaFunction): forward through
    ``tra_forward``, backward through ``tra_backward``; both on torch's
    current stream."""
    global _TRA_FUNCTION
    if _TRA_FUNCTION is None:
        import torch

        class TraFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, beta, p):
                ctx.save_for_backward(q, k, v)
                ctx.beta, ctx.p = float(beta), float(p)
                return tra_forward(q, k, v, beta, p)

            @staticmethod
            def backward(ctx, dout):
                q, k, v = ctx.saved_tensors
                dq, dk, dv = tra_backward(q, k, v, dout.to(q.dtype).contiguous(), ctx.beta, ctx.p)
                return dq, dk, dv, None, None

        _TRA_FUNCTION = TraFunction
    return _TRA_FUNCTION


def tra_attention(q, k, v, beta: float, p: float = 2.0):
    """Threshold rectified attention with autograd: ``tra_forward`` whose
    gradients with respect to q, k and v come from ``tra_backward`` (CUDA
    tensors ``[B, H, T, D]``, bfloat16 or float32)."""
    return _tra_function().apply(q, k, v, beta, p)


def tra_backward(q, k, v, dout, beta: float, p: float = 2.0, stream=None, deterministic: bool = False):
    """Gradients ``(dq, dk, dv)`` of the threshold rectified attention
    forward for the upstream gradient ``dout``; bf16 or fp32 CUDA tensors
    ``[B, H, T, D]``.  Scores are recomputed; runs on ``stream`` (default:
    torch's current stream) without synchronising.  bf16 runs the fused
    kernel (dq summed in fp32 in a run-dependent order) unless
    ``deterministic`` asks for the two-kernel form."""
    import torch

    if q.device.type != "cuda":
        raise BsaError("tra_backward takes CUDA tensors (no CPU path)")
    if not (q.shape == k.shape == v.shape == dout.shape) or q.dim() != 4:
        raise BsaError("q, k, v, dout must share one shape [B, H, T, D]", 2)
    if not (q.dtype == k.dtype == v.dtype == dout.dtype):
        raise BsaError("q, k, v, dout must share one dtype", 3)
    q, k, v, dout = q.contiguous(), k.contiguous(), v.contiguous(), dout.contiguous()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    B, H, T, D = q.shape
    st = tra_backward_ex_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(), dq.data_ptr(),
                             dk.data_ptr(), dv.data_ptr(), B, H, T, D, beta, p, _dtype_code(q),
                             BSA_TRA_BWD_DETERMINISTIC if deterministic else 0, _stream_handle(stream))
    _check(st, "tra_backward")
    return dq, dk, dv


def tra_diff_forward(q1, q2, k1, k2, v, beta: float, lam: float, p: float = 2.0, normalize: bool = True,
                     out=None, stream=None):
    """Threshold differential attention on bf16 CUDA tensors ``[B, H, T, D]``:
    ``TRA(n(q1), n(k1), v) - clamp(lam, 0, 1) * TRA(n(q2), n(k2), v)`` with
    ``n`` the row-wise L2 normalisation when ``normalize``."""
    import torch

    ts = (q1, q2, k1, k2, v)
    if q1.device.type != "cuda":
        raise BsaError("tra_diff_forward takes CUDA tensors (no CPU path)")
    if any(t.shape != q1.shape for t in ts) or q1.dim() != 4:
        raise BsaError("q1, q2, k1, k2, v must share one shape [B, H, T, D]", 2)
    if any(t.dtype != q1.dtype for t in ts):
        raise BsaError("q1, q2, k1, k2, v must share one dtype", 3)
    q1, q2, k1, k2, v = (t.contiguous() for t in ts)
    if out is None:
        out = torch.empty_like(q1)
    B, H, T, D = q1.shape
    st = tra_diff_forward_raw(q1.data_ptr(), q2.data_ptr(), k1.data_ptr(), k2.data_ptr(), v.data_ptr(),
                              out.data_ptr(), B, H, T, D, beta, lam, p, normalize, _dtype_code(q1),
                              _stream_handle(stream))
    _check(st, "tra_diff_forward")
    return out



def tra_diff_backward(q1, q2, k1, k2, v, dout, beta: float, lam: float, p: float = 2.0, normalize: bool = True,
                      want_dlam: bool = False, stream=None):
    """Gradients ``(dq1, dq2, dk1, dk2, dv, dlam)`` of ``tra_diff_forward`` for
    the upstream gradient ``dout`` (bf16 or fp32 CUDA tensors ``[B, H, T,
    D]``); ``dlam`` is a 1-element float32 CUDA tensor when ``want_dlam``,
    else None."""
    import torch

    ts = (q1, q2, k1, k2, v, dout)
    if q1.device.type != "cuda":
        raise BsaError("tra_diff_backward takes CUDA tensors (no CPU path)")
    if any(t.shape != q1.shape for t in ts) or q1.dim() != 4:
        raise BsaError("q1, q2, k1, k2, v, dout must share one shape [B, H, T, D]", 2)
    if any(t.dtype != q1.dtype for t in ts):
        raise BsaError("q1, q2, k1, k2, v, dout must share one dtype", 3)
    ts = tuple(t.contiguous() for t in ts)
    grads = tuple(torch.empty_like(q1) for _ in range(5))
    dlam = torch.empty(1, dtype=torch.float32, device=q1.device) if want_dlam else None
    B, H, T, D = q1.shape
    st = tra_diff_backward_raw(*(t.data_ptr() for t in ts), *(g.data_ptr() for g in grads),
                               dlam.data_ptr() if dlam is not None else None, B, H, T, D, beta, lam, p, normalize,
                               _dtype_code(q1), _stream_handle(stream))
    _check(st, "tra_diff_backward")
    return grads + (dlam,)


_TRA_DIFF_FUNCTION = None


def _tra_diff_function():
    """The autograd function of the differential form (page
    "triton_threshold_attention.py", differential_threshold_rela_triton):
    forward through ``tra_diff_forward``, backward through
    ``tra_diff_backward``; lambda may be a float or a 0-d / 1-element tensor
    (its gradient is returned when it requires one)."""
    global _TRA_DIFF_FUNCTION
    if _TRA_DIFF_FUNCTION is None:
        import torch

        class TraDiffFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q1, q2, k1, k2, v, beta, lam, p, normalize):
                lam_f = float(lam)
                ctx.save_for_backward(q1, q2, k1, k2, v)
                ctx.args = (float(beta), lam_f, float(p), bool(normalize))
                ctx.lam_tensor = isinstance(lam, torch.Tensor)
                return tra_diff_forward(q1, q2, k1, k2, v, beta, lam_f, p, normalize=normalize)

            @staticmethod
            def backward(ctx, dout):
                q1, q2, k1, k2, v = ctx.saved_tensors
                beta, lam, p, normalize = ctx.args
                want = ctx.lam_tensor and ctx.needs_input_grad[6]
                dq1, dq2, dk1, dk2, dv, dlam = tra_diff_backward(q1, q2, k1, k2, v, dout.to(q1.dtype), beta, lam, p,
                                                                 normalize, want_dlam=want)
                dl = dlam.reshape(()) if want else None
                return dq1, dq2, dk1, dk2, dv, None, dl, None, None

        _TRA_DIFF_FUNCTION = TraDiffFunction
    return _TRA_DIFF_FUNCTION


def tra_diff_attention(q1, q2, k1, k2, v, beta: float, lam, p: float = 2.0, normalize: bool = True):
    """Threshold differential attention with autograd: ``tra_diff_forward``
    whose gradients with respect to q1, q2, k1, k2, v (and lambda, when it is
    a tensor that requires one) come from ``tra_diff_backward``."""
    return _tra_diff_function().apply(q1, q2, k1, k2, v, beta, lam, p, normalize)

def nsa_select_forward(q, k, v, block_idx, block_size: int = 64, out=None, lse=None,
                       return_lse: bool = False, stream=None):
    """NSA selection-branch forward on CUDA tensors.

    q ``[B, Hq, T, D]``, k/v ``[B, Hkv, T, D]`` bf16, ``block_idx [B, Hkv, T,
    S]`` int32 (-1 = padding).  Returns ``out`` (and ``lse [B, Hq, T]`` fp32
    when ``return_lse``).
    """
    import torch

    if q.device.type != "cuda":
        raise BsaError("nsa_select_forward takes CUDA tensors (no CPU path)")
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or block_idx.dim() != 4:
        raise BsaError("q [B,Hq,T,D], k/v [B,Hkv,T,D], block_idx [B,Hkv,T,S] expected", 2)
    if not (q.dtype == k.dtype == v.dtype == torch.bfloat16):
        raise BsaError("nsa_select_forward takes bfloat16 q, k, v", 3)
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    S = block_idx.shape[-1]
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    idx = block_idx.to(torch.int32).contiguous()
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    st = nsa_select_forward_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(),
                                out.data_ptr(), lse.data_ptr() if lse is not None else None,
                                B, Hq, Hkv, T, D, block_size, S, _stream_handle(stream))
    _check(st, "nsa_select_forward")
    return (out, lse) if return_lse else out


def nsa_select_forward_fsa(q, k, v, block_idx, block_size: int = 64, out=None, lse=None,
                           return_lse: bool = False, workspace=None, stream=None):
    """NSA selection forward in the block-outer split-K form (same arguments
    and result as ``nsa_select_forward``).  ``workspace`` is a uint8 CUDA
    tensor of at least ``nsa_select_fsa_workspace_size(...)`` bytes; one is
    allocated when it is None.  It stays in use until the stream's work is
    done."""
    import torch

    if q.device.type != "cuda":
        raise BsaError("nsa_select_forward_fsa takes CUDA tensors (no CPU path)")
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or block_idx.dim() != 4:
        raise BsaError("q [B,Hq,T,D], k/v [B,Hkv,T,D], block_idx [B,Hkv,T,S] expected", 2)
    if not (q.dtype == k.dtype == v.dtype == torch.bfloat16):
        raise BsaError("nsa_select_forward_fsa takes bfloat16 q, k, v", 3)
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    S = block_idx.shape[-1]
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    idx = block_idx.to(torch.int32).contiguous()
    need = nsa_select_fsa_workspace_size(B, Hq, Hkv, T, D, block_size, S)
    if need == 0:
        raise BsaError("nsa_select_forward_fsa: sizes not accepted", 2)
    if workspace is None:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    st = nsa_select_forward_fsa_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(),
                                    lse.data_ptr() if lse is not None else None, B, Hq, Hkv, T, D, block_size, S,
                                    workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    _check(st, "nsa_select_forward_fsa")
    return (out, lse) if return_lse else out


def nsa_select_backward(q, k, v, block_idx, out, lse, dout, block_size: int = 64, workspace=None, stream=None):
    """Gradients ``(dq, dk, dv)`` of ``nsa_select_forward`` for the upstream
    gradient ``dout`` of its ``out``.

    q, out, dout ``[B, Hq, T, D]`` and k, v ``[B, Hkv, T, D]`` bf16,
    ``block_idx [B, Hkv, T, S]``, ``lse [B, Hq, T]`` fp32; ``out`` and ``lse``
    as the forward returned them.  The probabilities are recomputed from
    ``lse``; results repeat bit for bit.  ``workspace`` is a uint8 CUDA tensor
    of at least ``nsa_select_backward_workspace_size(...)`` bytes (allocated
    when None).  Runs on ``stream`` (default: torch's current stream) without
    synchronising.
    """
    import torch

    dev = _one_device("nsa_select_backward", q, k, v, block_idx, out, lse, dout, workspace)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, q.device, stream):
            return nsa_select_backward(q, k, v, block_idx, out, lse, dout, block_size, workspace)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or block_idx.dim() != 4:
        raise BsaError("q [B,Hq,T,D], k/v [B,Hkv,T,D], block_idx [B,Hkv,T,S] expected", 2)
    B, Hq, T, D = q.shape
    Hkv, S = k.shape[1], block_idx.shape[-1]
    if (q.shape != out.shape or q.shape != dout.shape or lse.shape != (B, Hq, T)
            or k.shape != (B, Hkv, T, D) or block_idx.shape != (B, Hkv, T, S)):
        raise BsaError("q, out, dout [B,Hq,T,D], lse [B,Hq,T], k/v [B,Hkv,T,D], block_idx [B,Hkv,T,S] expected", 2)
    if any(t.dtype != torch.bfloat16 for t in (q, k, v, out, dout)) or lse.dtype != torch.float32:
        raise BsaError("nsa_select_backward takes bfloat16 q, k, v, out, dout and float32 lse", 3)
    q, k, v, out, lse, dout = (t.contiguous() for t in (q, k, v, out, lse, dout))
    idx = _int32(torch, block_idx)
    if workspace is None:
        need = nsa_select_backward_workspace_size(B, Hq, Hkv, T, D, block_size, S)
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    elif not workspace.is_contiguous():  # (its elements are counted as its memory)
        raise BsaError("nsa_select_backward: workspace must be contiguous", 2)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    st = nsa_select_backward_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), out.data_ptr(),
                                 lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq,
                                 Hkv, T, D, block_size, S, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), torch.cuda.current_stream(dev).cuda_stream)
    _check(st, "nsa_select_backward")
    return dq, dk, dv


def _nsa_backward_counts(B, Hq, Hkv, T, S) -> bool:
    """Whether nsa_select_backward can count these sizes (the forward takes larger ones): rows and list entries are
    32-bit numbers, a query and its slot one of them, and (batch, kv head) pairs run along a grid's second axis."""
    return B * Hkv * T * S < 2 ** 31 and B * Hq * T < 2 ** 31 and T < 2 ** 26 and B * Hkv <= 65535


_NSA_FUNCTION = None


def _nsa_function():
    """The autograd function of the selection attention: forward through
    ``nsa_select_forward``, backward through ``nsa_select_backward``."""
    global _NSA_FUNCTION
    if _NSA_FUNCTION is None:
        import torch
        from torch.autograd.function import once_differentiable

        class NsaFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, block_idx, block_size):
                out, lse = nsa_select_forward(q, k, v, block_idx, block_size, return_lse=True)
                ctx.save_for_backward(q, k, v, block_idx, out, lse)
                ctx.block_size = int(block_size)
                return out

            @staticmethod
            @once_differentiable
            def backward(ctx, dout):
                q, k, v, block_idx, out, lse = ctx.saved_tensors
                dq, dk, dv = nsa_select_backward(q, k, v, block_idx, out, lse, dout.to(q.dtype), ctx.block_size)
                return dq, dk, dv, None, None

        _NSA_FUNCTION = NsaFunction
    return _NSA_FUNCTION


def nsa_select_attention(q, k, v, block_idx, block_size: int = 64):
    """NSA selection-branch attention with autograd: ``nsa_select_forward``
    whose gradients with respect to q, k and v come from
    ``nsa_select_backward`` (arguments as for ``nsa_select_forward``).  Runs on
    the current stream of the tensors' device, whichever device is current.
    Where a gradient is asked for, sizes that only the forward takes are refused
    here and not in the backward pass.  To capture a training step into a CUDA
    graph, capture forward and backward together, with no graph of the same
    leaves left from outside the capture.
    """
    import torch

    if (torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad)
            and q.dim() == k.dim() == block_idx.dim() == 4):
        sizes = (*q.shape[:2], k.shape[1], q.shape[2], block_idx.shape[3])
        if not _nsa_backward_counts(*sizes):
            raise BsaError(f"nsa_select_attention: no gradients for B, Hq, Hkv, T, S = {sizes} "
                           "(the limits of nsa_select_backward)", 2)
    with torch.cuda.device(_one_device("nsa_select_attention", q, k, v, block_idx)):
        return _nsa_function().apply(q, k, v, block_idx, block_size)


def _check_cache(torch, what, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, B, Hkv, D):
    """Shapes and types of the paged cache; returns (num_pages, page_size, max_pages)."""
    if k_cache.dim() != 4 or page_table.dim() != 2 or page_table.shape[0] != B or cache_lens.shape != (B,):
        raise BsaError(f"{what}: k_cache [pages,Hkv,page_size,D], page_table [B,max_pages], cache_lens [B] expected", 2)
    pages, _, page_size, _ = shape = k_cache.shape
    if not (shape[1] == Hkv and shape[3] == D and v_cache.shape == shape and k_scale.shape == (pages, Hkv)
            and v_scale.shape == k_scale.shape and k_cache.dtype in (torch.uint8, torch.float8_e4m3fn)
            and v_cache.dtype in (torch.uint8, torch.float8_e4m3fn) and k_scale.dtype is torch.float32
            and v_scale.dtype is torch.float32 and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_scale.is_contiguous() and v_scale.is_contiguous()):  # (all of it at once: half the time)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            _in_place(what, name, t, (pages, Hkv, page_size, D), torch.float8_e4m3fn, torch.uint8)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _in_place(what, name, t, (pages, Hkv), torch.float32)
    return pages, page_size, page_table.shape[1]


def nsa_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens=None, inv_freq=None,
                     interleaved: bool = False, q=None, q_out=None, stream=None):
    """Writes the keys and values of new tokens into a paged e4m3 cache, in
    place, keys rotated by position on the way.

    k, v ``[B, Hkv, n, D]`` bf16 or fp32; ``k_cache``/``v_cache [pages, Hkv,
    page_size, D]`` float8_e4m3fn (or uint8 codes), ``k_scale``/``v_scale
    [pages, Hkv]`` fp32, ``page_table [B, max_pages]``; ``cache_lens [B]``
    counts the tokens held before (it is not advanced here), ``new_lens [B]``
    the new ones of each sequence (default n).  ``inv_freq [rotary_dim / 2]``
    gives the rotation's angle per position of each pair, halves apart or
    neighbours if ``interleaved`` (None: no rotation).  With ``q [B, Hq, n,
    D]`` the rotated queries are returned, in ``q_out`` if given (q itself is
    allowed; rows past ``new_lens`` are left as they were, or zero in a new
    tensor).  Has no gradient: where autograd records, tensors that require one
    are refused.  Runs on ``stream`` (default: torch's current stream) without
    synchronising.
    """
    import torch

    what = "nsa_cache_append"
    if torch.is_grad_enabled():
        _no_gradient(what, k, v, q, q_out, k_cache, v_cache, k_scale, v_scale, inv_freq)
    dev = _one_device(what, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens, inv_freq, q,
                      q_out)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, k.device, stream):
            return nsa_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens,
                                    inv_freq, interleaved, q, q_out)
    if k.dim() != 4 or k.shape != v.shape or (q is not None and q.dim() != 4):
        raise BsaError("k, v [B,Hkv,n,D] and q [B,Hq,n,D] expected", 2)
    B, Hkv, n, D = k.shape
    Hq = Hkv if q is None else q.shape[1]
    pages, page_size, max_pages = _check_cache(torch, what, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens,
                                               B, Hkv, D)
    if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise BsaError("k, v, q must share one dtype", 3)
    if q is not None and q.shape != (B, Hq, n, D):
        raise BsaError("q must be [B,Hq,n,D] with k's B, n and D", 2)
    if q is None and q_out is not None:
        raise BsaError("q_out given without q")
    if q_out is not None:
        _in_place(what, "q_out", q_out, q.shape, q.dtype)
    if new_lens is not None and new_lens.shape != (B,):
        raise BsaError("new_lens must be [B]", 2)
    if inv_freq is not None and inv_freq.dim() != 1:
        raise BsaError("inv_freq must be [rotary_dim / 2]", 2)
    rotary = 0 if inv_freq is None else 2 * inv_freq.numel()
    k, v = k.contiguous(), v.contiguous()
    table, lens = _int32(torch, page_table), _int32(torch, cache_lens)
    news = None if new_lens is None else _int32(torch, new_lens)
    freq = None if inv_freq is None else inv_freq.to(torch.float32).contiguous()
    q_ptr = out_ptr = None
    written = [k_cache, v_cache, k_scale, v_scale]
    if q is not None:
        if q_out is not None:
            written.append(q_out)
        else:
            make = torch.empty if news is None else torch.zeros
            q_out = make(q.shape, dtype=q.dtype, device=q.device)
        q = q.contiguous()
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    st = nsa_cache_append_raw(k.data_ptr(), v.data_ptr(), q_ptr, out_ptr, k_cache.data_ptr(), v_cache.data_ptr(),
                              k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(), lens.data_ptr(),
                              None if news is None else news.data_ptr(), None if freq is None else freq.data_ptr(), B,
                              Hq, Hkv, n, D, page_size, max_pages, pages, rotary, interleaved, _dtype_code(k),
                              torch.cuda.current_stream(dev).cuda_stream)
    _check(st, what)
    torch.autograd.graph.increment_version(written)  # a graph that saved one of them must not use it any more
    return q_out


def nsa_select_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx=None, out=None,
                      lse=None, return_lse: bool = False, workspace=None, stream=None):
    """``nsa_select_forward`` for the last token of each sequence, over the
    paged e4m3 cache that ``nsa_cache_append`` fills.

    q ``[B, Hq, 1, D]`` bf16 (rotated), the cache as for ``nsa_cache_append``,
    ``cache_lens [B]`` with the query's own token counted; ``block_idx [B,
    Hkv, 1, S]``, S from 1 to 32, lists logical pages (a set, -1 = padding), None
    reads every page.  Returns ``out [B, Hq, 1, D]`` (and ``lse [B, Hq, 1]`` fp32 when
    ``return_lse``); an empty sequence or selection gives 0 and -1e9.
    ``workspace`` is a uint8 CUDA tensor of at least
    ``nsa_select_decode_workspace_size(...)`` bytes (allocated when None).
    Has no gradient: where autograd records, tensors that require one are
    refused.  Runs on ``stream`` (default: torch's current stream) without
    synchronising.
    """
    import torch

    what = "nsa_select_decode"
    if torch.is_grad_enabled():
        _no_gradient(what, q, k_cache, v_cache, k_scale, v_scale, out, lse)
    dev = _one_device(what, q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx, out, lse,
                      workspace)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, q.device, stream):
            return nsa_select_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx, out,
                                     lse, return_lse, workspace)
    if q.dim() != 4 or q.shape[2] != 1 or k_cache.dim() != 4:
        raise BsaError("q [B,Hq,1,D] and k_cache [pages,Hkv,page_size,D] expected", 2)
    if q.dtype != torch.bfloat16:
        raise BsaError("nsa_select_decode takes bfloat16 q", 3)
    B, Hq, _, D = q.shape
    Hkv = k_cache.shape[1]
    pages, page_size, max_pages = _check_cache(torch, what, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens,
                                               B, Hkv, D)
    S = 0
    if block_idx is not None:
        S = block_idx.shape[-1] if block_idx.dim() == 4 else 0
        if block_idx.shape != (B, Hkv, 1, S) or not 0 < S <= 32:  # (an empty one has no address: none, to the library)
            raise BsaError("block_idx must be [B,Hkv,1,S] with S from 1 to 32", 2)
    written = []
    if out is not None:
        _in_place(what, "out", out, q.shape, torch.bfloat16)
        written.append(out)
    if lse is not None:
        _in_place(what, "lse", lse, (B, Hq, 1), torch.float32)
        written.append(lse)
    q = q.contiguous()
    table, lens = _int32(torch, page_table), _int32(torch, cache_lens)
    idx = None if block_idx is None else _int32(torch, block_idx)
    if workspace is None:
        need = nsa_select_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S)
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    elif not workspace.is_contiguous():
        raise BsaError(f"{what}: workspace must be contiguous", 2)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, 1), device=q.device, dtype=torch.float32)
    st = nsa_select_decode_raw(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                               v_scale.data_ptr(), table.data_ptr(), lens.data_ptr(),
                               None if idx is None else idx.data_ptr(), out.data_ptr(),
                               None if lse is None else lse.data_ptr(), B, Hq, Hkv, D, page_size, max_pages, pages, S,
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               torch.cuda.current_stream(dev).cuda_stream)
    _check(st, what)
    if written:
        torch.autograd.graph.increment_version(written)
    return (out, lse) if return_lse else out


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: int = 0, fast: float = 32.0, slow: float = 1.0, device=None):
    """``(inv_freq, rotary_scale)`` of a rotation over ``rotary_dim`` elements, for ``qk_norm_rope`` and the cache
    appends: ``base ** (-2 j / rotary_dim)``, for contexts ``factor`` times as long as the ``original_length`` of
    training scaled by

    * ``"linear"``: every frequency over ``factor``;
    * ``"base"``: the base times ``factor ** (r / (r - 2))``, which leaves the fastest pair and divides the slowest;
    * ``"bands"``: pairs that make more than ``fast`` turns over ``original_length`` as they are, those under ``slow``
      turns over ``factor``, those between in proportion to their turns, and ``rotary_scale = 0.1 ln(factor) + 1``.
      Checkpoints differ in both: some take the pairs between in proportion to their index j, whose frequencies a
      caller makes for itself, and some use no factor on attention: leave ``rotary_scale`` at 1 for those.

    ``inv_freq`` is float32, ``rotary_scale`` a number (1 but for ``"bands"``).
    """
    import math

    import torch

    if rotary_dim < 2 or rotary_dim % 2 or not base > 1.0 or not factor >= 1.0:
        raise BsaError("rope_frequencies: an even rotary_dim, base > 1 and factor >= 1 expected", 2)
    if scaling not in ("none", "linear", "base", "bands"):
        raise BsaError(f"rope_frequencies: unknown scaling {scaling!r}", 4)
    if scaling == "base" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if original_length < 1 or not fast > slow:
            raise BsaError("rope_frequencies: bands need original_length and fast > slow", 2)
        keep = ((f * original_length / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    return f.to(device=device, dtype=torch.float32), scale


def _row_strides(t):
    """``t`` [B, H, T, D] as the kernels read rows in place, and its (batch, head, token) strides; a copy where a row's
    elements do not follow each other or do not start on a 16-byte boundary."""
    sb, sh, st, sd = t.stride()
    nb, nh, nt, _ = t.shape
    if nb == 1:
        sb = 0
    if nh == 1:
        sh = 0
    if nt == 1:
        st = 0
    if sd != 1 or (sb | sh | st) % (16 // t.element_size()) or t.data_ptr() % 16:
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
        sb, sh, st, _ = t.stride()
    return t, (sb, sh, st)


def _rows_like(torch, t):
    """An empty tensor of ``t``'s shape, heads inside tokens where t's are (so a projection's gradient is as it was)."""
    if t.stride(1) < t.stride(2):
        return torch.empty((t.shape[0], t.shape[2], t.shape[1], t.shape[3]), dtype=t.dtype,
                           device=t.device).transpose(1, 2)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _aligned(t):
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _row_parameters(torch, what, q_weight, k_weight, inv_freq, D):
    """Weights of one dtype and frequencies as the kernels take them; (q_weight, k_weight, their dtype, inv_freq)."""
    kind = BSA_F32
    if q_weight is not None or k_weight is not None:
        types = []
        for w in (q_weight, k_weight):
            if w is not None:
                if w.shape != (D,):
                    raise BsaError(f"{what}: weights must be [{D}]", 2)
                types.append(w.dtype)
        if types[0] is types[-1] is torch.bfloat16:
            kind = BSA_BF16
        elif not (types[0] is types[-1] is torch.float32):
            if any(x not in (torch.bfloat16, torch.float32) for x in types):
                raise BsaError(f"{what}: weights must be float32 or bfloat16", 3)
            q_weight, k_weight = q_weight.to(torch.float32), k_weight.to(torch.float32)
        if q_weight is not None and (q_weight.data_ptr() % 16 or not q_weight.is_contiguous()):
            q_weight = _aligned(q_weight.contiguous())
        if k_weight is not None and (k_weight.data_ptr() % 16 or not k_weight.is_contiguous()):
            k_weight = _aligned(k_weight.contiguous())
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise BsaError(f"{what}: inv_freq must be [rotary_dim / 2]", 2)
        if inv_freq.dtype is not torch.float32 or inv_freq.data_ptr() % 16 or not inv_freq.is_contiguous():
            inv_freq = _aligned(inv_freq.to(torch.float32).contiguous())
        if not inv_freq.numel():
            inv_freq = None
    return q_weight, k_weight, kind, inv_freq


def _row_inputs(torch, what, q, k, q_weight, k_weight, inv_freq, positions):
    """Checks of ``qk_norm_rope``'s inputs; (q_weight, k_weight, their dtype, inv_freq, positions)."""
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4 or qs[0] != ks[0] or qs[2:] != ks[2:]:
        raise BsaError(f"{what}: q [B,Hq,T,D] and k [B,Hkv,T,D] expected", 2)
    if q.dtype is not k.dtype:
        raise BsaError(f"{what}: q and k must share one dtype", 3)
    if positions is not None:
        shape = (qs[0], qs[2])
        if positions.shape != shape:
            if positions.shape != shape[1:]:
                raise BsaError(f"{what}: positions must be [B,T] or [T]", 2)
            positions = positions.expand(shape)
        positions = _int32(torch, positions)
    return (*_row_parameters(torch, what, q_weight, k_weight, inv_freq, qs[3]), positions)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(torch, dev):
    """The handle of the device's current stream (without a stream object around it, which takes a microsecond)."""
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(dev).cuda_stream if get is None else get(dev)


def qk_norm_rope_forward(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, interleaved: bool = False,
                         rotary_scale: float = 1.0, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and its rotation by position, in
    one pass: ``(q_out [B, Hq, T, D], k_out [B, Hkv, T, D])``, contiguous, for
    the attention calls.

    q, k bf16 or fp32, read in place by their strides (views of a fused
    projection ``[B, T, heads, D]`` among them).  ``q_weight``/``k_weight [D]``
    (None: that one is not normalised), ``inv_freq [rotary_dim / 2]`` (None: no
    rotation; ``rope_frequencies`` makes them) with pairs halves apart or
    neighbours if ``interleaved``, ``positions [B, T]`` or ``[T]`` (None: 0 ..
    T - 1); the rotated elements are multiplied by ``rotary_scale``.  Arithmetic
    is fp32, rounded once.  ``q_out``/``k_out`` (None: new ones) may be q and k
    themselves where these are contiguous; memory that meets another tensor's
    is refused.  Where autograd records, tensors that require a
    gradient are refused: ``qk_norm_rope`` has one.  Runs on ``stream`` (default:
    torch's current stream) without synchronising.
    """
    import torch

    what = "qk_norm_rope_forward"
    if torch.is_grad_enabled():
        _no_gradient(what, q, k, q_weight, k_weight, inv_freq, q_out, k_out)
    dev = _one_device(what, q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, q.device, stream):
            return qk_norm_rope_forward(q, k, q_weight, k_weight, inv_freq, positions, interleaved, rotary_scale, eps,
                                        q_out, k_out)
    qw, kw, kind, freq, pos = _row_inputs(torch, what, q, k, q_weight, k_weight, inv_freq, positions)
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    written = None
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _in_place(what, "q_out", q_out, q.shape, q.dtype)
        written = [q_out]
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    else:
        _in_place(what, "k_out", k_out, k.shape, k.dtype)
        written = [*(written or ()), k_out]
    (q, qs), (k, ks) = _row_strides(q), _row_strides(k)
    if written:
        _apart(what, "q_out", q_out, q, k, k_out, qw, kw, pos, freq)
        _apart(what, "k_out", k_out, k, q, qw, kw, pos, freq)
    row = T * D
    st = qk_norm_rope_forward_raw(
        q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), _ptr(qw), _ptr(kw), _ptr(pos), _ptr(freq),
        (*qs, *ks, Hq * row, row, D, Hkv * row, row, D), B, Hq, Hkv, T, D,
        0 if freq is None else 2 * freq.numel(), interleaved, rotary_scale, eps, _dtype_code(q), kind,
        _raw_stream(torch, dev))
    if st:
        _check(st, what)
    if written:
        torch.autograd.graph.increment_version(written)
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, inv_freq=None, positions=None,
                          interleaved: bool = False, rotary_scale: float = 1.0, eps: float = 1e-6, workspace=None,
                          stream=None):
    """Gradients ``(dq, dk, dq_weight, dk_weight)`` of ``qk_norm_rope_forward``
    for the upstream gradients ``dq_out``, ``dk_out`` of its results.

    Arguments as for the forward; dq and dk lie in memory as q and k do (heads
    inside tokens, or tokens inside heads), the weights' gradients are fp32
    (None without weights).  Results repeat bit for bit.  ``workspace`` is a
    uint8 CUDA tensor of at least ``qk_norm_rope_backward_workspace_size(...)``
    bytes (allocated when None).  Runs on ``stream`` (default: torch's current
    stream) without synchronising.
    """
    import torch

    what = "qk_norm_rope_backward"
    dev = _one_device(what, q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, positions, workspace)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, q.device, stream):
            return qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, positions, interleaved,
                                         rotary_scale, eps, workspace)
    qw, kw, kind, freq, pos = _row_inputs(torch, what, q, k, q_weight, k_weight, inv_freq, positions)
    if dq_out.shape != q.shape or dk_out.shape != k.shape:
        raise BsaError(f"{what}: dq_out and dk_out must have the shapes of q and k", 2)
    if dq_out.dtype != q.dtype or dk_out.dtype != k.dtype:
        raise BsaError(f"{what}: dq_out and dk_out must have the dtype of q and k", 3)
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    if workspace is None:
        workspace = torch.empty(max(qk_norm_rope_backward_workspace_size(B, Hq, Hkv, T, D), 1), device=q.device,
                                dtype=torch.uint8)
    elif not workspace.is_contiguous():
        raise BsaError(f"{what}: workspace must be contiguous", 2)
    dq, dk = _rows_like(torch, q), _rows_like(torch, k)
    dqw, dkw = (None if w is None else torch.empty(D, dtype=torch.float32, device=q.device) for w in (qw, kw))
    (q, s0), (k, s1), (dq_out, s2), (dk_out, s3) = (_row_strides(t) for t in (q, k, dq_out, dk_out))
    st = qk_norm_rope_backward_raw(
        q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), _ptr(dqw),
        _ptr(dkw), _ptr(qw), _ptr(kw), _ptr(pos), _ptr(freq),
        (*s0, *s1, *s2, *s3, *dq.stride()[:3], *dk.stride()[:3]), B, Hq, Hkv, T, D,
        0 if freq is None else 2 * freq.numel(), interleaved, rotary_scale, eps, _dtype_code(q), kind,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _raw_stream(torch, dev))
    if st:
        _check(st, what)
    return dq, dk, dqw, dkw


_ROPE_FUNCTION = None


def _rope_function():
    """The autograd function of the norm and rotation of query and key heads."""
    global _ROPE_FUNCTION
    if _ROPE_FUNCTION is None:
        import torch
        from torch.autograd.function import once_differentiable

        class QkNormRopeFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, q_weight, k_weight, inv_freq, positions, interleaved, rotary_scale, eps):
                ctx.save_for_backward(q, k, q_weight, k_weight, inv_freq, positions)
                ctx.rest = bool(interleaved), float(rotary_scale), float(eps)
                return qk_norm_rope_forward(q, k, q_weight, k_weight, inv_freq, positions, *ctx.rest)

            @staticmethod
            @once_differentiable
            def backward(ctx, dq_out, dk_out):
                q, k, q_weight, k_weight, inv_freq, positions = ctx.saved_tensors
                dq, dk, dqw, dkw = qk_norm_rope_backward(q, k, dq_out.to(q.dtype), dk_out.to(k.dtype), q_weight,
                                                         k_weight, inv_freq, positions, *ctx.rest)
                dqw = None if dqw is None else dqw.to(q_weight.dtype)
                dkw = None if dkw is None else dkw.to(k_weight.dtype)
                return dq, dk, dqw, dkw, None, None, None, None, None

        _ROPE_FUNCTION = QkNormRopeFunction
    return _ROPE_FUNCTION


def qk_norm_rope(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, interleaved: bool = False,
                 rotary_scale: float = 1.0, eps: float = 1e-6):
    """``qk_norm_rope_forward`` with autograd: gradients with respect to q, k
    and the weights come from ``qk_norm_rope_backward`` (frequencies have
    none).  Runs on the current stream of the tensors' device, whichever
    device is current.  To capture a training step into a CUDA graph, capture
    forward and backward together, with no graph of the same leaves left from
    outside the capture.
    """
    import torch

    if torch.is_grad_enabled():
        _no_gradient("qk_norm_rope with respect to inv_freq", inv_freq)
    with torch.cuda.device(_one_device("qk_norm_rope", q, k, q_weight, k_weight, inv_freq, positions)):
        return _rope_function().apply(q, k, q_weight, k_weight, inv_freq, positions, interleaved, rotary_scale, eps)


def _check_cache4(torch, what, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table, cache_lens, B, Hkv,
                  D):
    """Shapes and types of the paged 4-bit cache; returns (num_pages, page_size, max_pages)."""
    shape, table = k_cache.shape, page_table.shape
    if len(shape) != 4 or len(table) != 2 or table[0] != B or cache_lens.shape != (B,):
        raise BsaError(f"{what}: k_cache [pages,Hkv,page_size,D/2], page_table [B,max_pages], cache_lens [B] expected",
                       2)
    pages, _, page_size, _ = shape
    codes, scales = (pages, Hkv, page_size, D // 2), (pages, Hkv, page_size, D // 16)
    kinds = torch.float8_e4m3fn, torch.uint8
    if not (shape == codes == v_cache.shape and k_scale.shape == scales and v_scale.shape == scales
            and k_cache.dtype is v_cache.dtype is torch.uint8 and k_scale.dtype in kinds and v_scale.dtype in kinds
            and k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous()
            and v_scale.is_contiguous()):
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            _in_place(what, name, t, codes, torch.uint8)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _in_place(what, name, t, scales, *kinds)
    if k_factor is not None:
        _in_place(what, "k_factor", k_factor, (Hkv,), torch.float32)
    if v_factor is not None:
        _in_place(what, "v_factor", v_factor, (Hkv,), torch.float32)
    return pages, page_size, table[1]


def nsa_cache4_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens=None, inv_freq=None,
                      interleaved: bool = False, q=None, q_out=None, q_weight=None, k_weight=None,
                      rotary_scale: float = 1.0, eps: float = 1e-6, k_factor=None, v_factor=None, stream=None):
    """Writes the keys and values of new tokens into a paged cache of 4-bit
    codes, in place, keys normalised and rotated by position on the way.

    As ``nsa_cache_append`` but for the cache: ``k_cache``/``v_cache [pages,
    Hkv, page_size, D / 2]`` uint8 (two e2m1 codes a byte, the first in the low
    half), ``k_scale``/``v_scale [pages, Hkv, page_size, D / 16]`` float8_e4m3fn
    (or uint8 codes): a scale for every 16 elements of a token; and
    ``k_factor``/``v_factor [Hkv]`` fp32, optional factors of the heads, the same
    in every call on a cache.  k, v and q are read in place by their strides;
    ``q_weight``/``k_weight [D]`` (None: not normalised), ``rotary_scale`` and
    ``eps`` are those of ``qk_norm_rope_forward``.  Returns the queries,
    normalised and rotated (None without q).  Has no gradient: where autograd
    records, tensors that require one are refused.  Runs on ``stream`` (default:
    torch's current stream) without synchronising.
    """
    import torch

    what = "nsa_cache4_append"
    if torch.is_grad_enabled():
        _no_gradient(what, k, v, q, q_out, k_scale, v_scale, inv_freq, q_weight, k_weight, k_factor, v_factor)
    dev = _one_device(what, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens, inv_freq, q,
                      q_out, q_weight, k_weight, k_factor, v_factor)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, k.device, stream):
            return nsa_cache4_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens,
                                     inv_freq, interleaved, q, q_out, q_weight, k_weight, rotary_scale, eps, k_factor,
                                     v_factor)
    if k.dim() != 4 or k.shape != v.shape or (q is not None and q.dim() != 4):
        raise BsaError("k, v [B,Hkv,n,D] and q [B,Hq,n,D] expected", 2)
    B, Hkv, n, D = k.shape
    Hq = Hkv if q is None else q.shape[1]
    pages, page_size, max_pages = _check_cache4(torch, what, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor,
                                                page_table, cache_lens, B, Hkv, D)
    if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise BsaError("k, v, q must share one dtype", 3)
    if q is not None and q.shape != (B, Hq, n, D):
        raise BsaError("q must be [B,Hq,n,D] with k's B, n and D", 2)
    if q is None and (q_out is not None or q_weight is not None):
        raise BsaError("q_out or q_weight given without q")
    if q_out is not None:
        _in_place(what, "q_out", q_out, q.shape, q.dtype)
    if new_lens is not None and new_lens.shape != (B,):
        raise BsaError("new_lens must be [B]", 2)
    qw, kw, kind, freq = _row_parameters(torch, what, q_weight, k_weight, inv_freq, D)
    (k, ks), (v, vs) = _row_strides(k), _row_strides(v)
    qs = (0, 0, 0)
    table, lens = _int32(torch, page_table), _int32(torch, cache_lens)
    news = None if new_lens is None else _int32(torch, new_lens)
    written = [k_cache, v_cache, k_scale, v_scale]
    if q is not None:
        if q_out is not None:
            written.append(q_out)
        else:
            make = torch.empty if news is None else torch.zeros
            q_out = make(q.shape, dtype=q.dtype, device=q.device)
        q, qs = _row_strides(q)
    st = nsa_cache4_append_raw(
        k.data_ptr(), v.data_ptr(), _ptr(q), _ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), _ptr(k_factor), _ptr(v_factor), table.data_ptr(), lens.data_ptr(), _ptr(news), _ptr(qw),
        _ptr(kw), _ptr(freq), (*ks, *vs, *qs), B, Hq, Hkv, n, D, page_size, max_pages, pages,
        0 if freq is None else 2 * freq.numel(), interleaved, rotary_scale, eps, _dtype_code(k), kind,
        _raw_stream(torch, dev))
    if st:
        _check(st, what)
    torch.autograd.graph.increment_version(written)  # a graph that saved one of them must not use it any more
    return q_out


def nsa_cache4_read(k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, n: int, starts=None, k_factor=None,
                    v_factor=None, dtype=None, k_out=None, v_out=None, stream=None):
    """The values that the 4-bit cache holds of tokens ``starts[b] + i``, ``i <
    n`` (``starts`` None: the first n): ``(k, v)``, each ``[B, Hkv, n, D]`` of
    ``dtype`` (bf16 or fp32; default bf16, or that of ``k_out``).

    The cache, its factors and ``cache_lens`` as ``nsa_cache4_append`` left
    them, the new tokens counted.  Rows past a sequence's length are zero.
    ``k_out`` and ``v_out``, given together, overlap nothing else.  Runs on
    ``stream`` (default: torch's current stream) without synchronising.
    """
    import torch

    what = "nsa_cache4_read"
    if torch.is_grad_enabled():
        _no_gradient(what, k_scale, v_scale, k_factor, v_factor, k_out, v_out)
    dev = _one_device(what, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, starts, k_factor, v_factor,
                      k_out, v_out)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, k_cache.device, stream):
            return nsa_cache4_read(k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, n, starts, k_factor,
                                   v_factor, dtype, k_out, v_out)
    if k_cache.dim() != 4 or page_table.dim() != 2:
        raise BsaError("k_cache [pages,Hkv,page_size,D/2] and page_table [B,max_pages] expected", 2)
    B, Hkv, D = page_table.shape[0], k_cache.shape[1], 2 * k_cache.shape[3]
    pages, page_size, max_pages = _check_cache4(torch, what, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor,
                                                page_table, cache_lens, B, Hkv, D)
    if starts is not None and starts.shape != (B,):
        raise BsaError("starts must be [B]", 2)
    if (k_out is None) != (v_out is None):
        raise BsaError(f"{what}: give k_out and v_out together")
    if dtype is None:
        dtype = torch.bfloat16 if k_out is None else k_out.dtype
    shape, written = (B, Hkv, n, D), []
    if k_out is not None:
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            _in_place(what, name, t, shape, dtype)
            written.append(t)
    else:
        if n < 1:
            raise BsaError(f"{what}: n must be at least 1", 2)
        k_out, v_out = (torch.empty(shape, dtype=dtype, device=k_cache.device) for _ in range(2))
    table, lens = _int32(torch, page_table), _int32(torch, cache_lens)
    begin = None if starts is None else _int32(torch, starts)
    if written:
        cache = k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, table, lens, begin
        _apart(what, "k_out", k_out, None, v_out, *cache)
        _apart(what, "v_out", v_out, None, *cache)
    st = nsa_cache4_read_raw(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _ptr(k_factor), _ptr(v_factor),
        table.data_ptr(), _ptr(begin), lens.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), B, Hkv, n, D, page_size,
        max_pages, pages, _dtype_code(k_out), _raw_stream(torch, dev))
    if st:
        _check(st, what)
    if written:
        torch.autograd.graph.increment_version(written)
    return k_out, v_out


def nsa_cache4_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx=None, k_factor=None,
                      v_factor=None, out=None, lse=None, return_lse: bool = False, workspace=None, stream=None):
    """``nsa_select_decode`` over the paged 4-bit cache that
    ``nsa_cache4_append`` fills.

    q ``[B, Hq, 1, D]`` bf16 (normalised and rotated), the cache and its factors
    as for ``nsa_cache4_append``, everything else as for ``nsa_select_decode``
    (``workspace``: ``nsa_cache4_decode_workspace_size(...)`` bytes; selected
    pages use none).
    """
    import torch

    what = "nsa_cache4_decode"
    if torch.is_grad_enabled():
        _no_gradient(what, q, k_scale, v_scale, k_factor, v_factor, out, lse)
    dev = _one_device(what, q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx, k_factor,
                      v_factor, out, lse, workspace)
    if stream is not None or dev != torch.cuda.current_device():
        with _on_stream(torch, q.device, stream):
            return nsa_cache4_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx,
                                     k_factor, v_factor, out, lse, return_lse, workspace)
    if q.dim() != 4 or q.shape[2] != 1 or k_cache.dim() != 4:
        raise BsaError("q [B,Hq,1,D] and k_cache [pages,Hkv,page_size,D/2] expected", 2)
    if q.dtype != torch.bfloat16:
        raise BsaError("nsa_cache4_decode takes bfloat16 q", 3)
    B, Hq, _, D = q.shape
    Hkv = k_cache.shape[1]
    pages, page_size, max_pages = _check_cache4(torch, what, k_cache, v_cache, k_scale, v_scale, k_factor, v_factor,
                                                page_table, cache_lens, B, Hkv, D)
    S = 0
    if block_idx is not None:
        S = block_idx.shape[-1] if block_idx.dim() == 4 else 0
        if block_idx.shape != (B, Hkv, 1, S) or not 0 < S <= 32:  # (an empty one has no address: none, to the library)
            raise BsaError("block_idx must be [B,Hkv,1,S] with S from 1 to 32", 2)
    written = []
    if out is not None:
        _in_place(what, "out", out, q.shape, torch.bfloat16)
        written.append(out)
    if lse is not None:
        _in_place(what, "lse", lse, (B, Hq, 1), torch.float32)
        written.append(lse)
    q = _aligned(q.contiguous())
    table, lens = _int32(torch, page_table), _int32(torch, cache_lens)
    idx = None if block_idx is None else _int32(torch, block_idx)
    space = 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise BsaError(f"{what}: workspace must be contiguous", 2)
        space = workspace.numel() * workspace.element_size()
    elif block_idx is None:  # (selected pages need none)
        space = max(nsa_cache4_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S), 1)
        workspace = torch.empty(space, device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, 1), device=q.device, dtype=torch.float32)
    st = nsa_cache4_decode_raw(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _ptr(k_factor),
        _ptr(v_factor), table.data_ptr(), lens.data_ptr(), _ptr(idx), out.data_ptr(), _ptr(lse), B, Hq, Hkv, D,
        page_size, max_pages, pages, S, _ptr(workspace), space, _raw_stream(torch, dev))
    if st:
        _check(st, what)
    if written:
        torch.autograd.graph.increment_version(written)
    return (out, lse) if return_lse else out


def selftest_wait_timeout(limit_cycles: int = 100000, stream=None) -> int:
    """Run the bounded-wait expiry self test (a wait on an mbarrier nothing
    arrives on, with a short limit).  Returns the kernel's result word: 0 when
    the wait gave up as designed.  The timeout is also recorded in the device
    error word that ``device_error()`` reads and clears."""
    import torch

    res = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    _check(load_library().bsa_selftest_wait_timeout(int(limit_cycles), res.data_ptr(), _stream_handle(stream)),
           "bsa_selftest_wait_timeout")
    return int(res.item())


def selftest_log2(x, stream=None):
    """The epilogue's FMA-pipe log2 and CUDA's log2f on the same float32
    device tensor; returns ``(y_fma, y_ref)``."""
    import torch

    if not (x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()):
        raise BsaError("selftest_log2 needs a contiguous float32 CUDA tensor")
    y_fma, y_ref = torch.empty_like(x), torch.empty_like(x)
    _check(load_library().bsa_selftest_log2(x.data_ptr(), y_fma.data_ptr(), y_ref.data_ptr(), x.numel(),
                                            _stream_handle(stream)), "bsa_selftest_log2")
    return y_fma, y_ref


def selftest_exp2(y, stream=None):
    """The epilogue's FMA-pipe exp2 (fp32, before the bf16 rounding) and
    CUDA's exp2f on the same float32 device tensor; returns ``(w_fma, w_ref)``."""
    import torch

    if not (y.is_cuda and y.dtype == torch.float32 and y.is_contiguous()):
        raise BsaError("selftest_exp2 needs a contiguous float32 CUDA tensor")
    w_fma, w_ref = torch.empty_like(y), torch.empty_like(y)
    _check(load_library().bsa_selftest_exp2(y.data_ptr(), w_fma.data_ptr(), w_ref.data_ptr(), y.numel(),
                                            _stream_handle(stream)), "bsa_selftest_exp2")
    return w_fma, w_ref


def read_probe(buf, reps: int, sink, stream=None):
    """Enqueue the streaming-read probe over the bytes of CUDA tensor ``buf``
    (``reps`` passes); ``sink`` is a 1-element int32 CUDA tensor."""
    nbytes = buf.numel() * buf.element_size()
    _check(load_library().bsa_read_probe(buf.data_ptr(), nbytes - nbytes % 16, int(reps), sink.data_ptr(),
                                         _stream_handle(stream)), "bsa_read_probe")
