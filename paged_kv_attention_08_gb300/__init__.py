"""Paged-attention decode for GB300 (sm_103a): thin Python binding.

Every call marshals torch tensors into the C ABI of ``libpa_decode.so``
(declared in ``include/pa_decode.h``) and launches on the current torch CUDA
stream.  Torch supplies device memory and streams only; all arithmetic runs in
the library's CUDA kernels.  There is no fallback: if the library is not built
or a call is rejected, an exception is raised.

    decode(out, q, k_cache, v_cache, block_tables, context_lens, scale)
    decode_splitkv(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                   max_context_len, partition_tokens=0, workspace=None)
    decode_splitkv_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                           max_context_len, partition_tokens=0)
    decode_multi(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                 max_context_len, partition_tokens=0, workspace=None)
    append_kv(k_cache, v_cache, k_new, v_new, block_tables, positions)
    rope_phases(inv_freq)
    rope_append_kv(q_out, k_cache, v_cache, q, k_new, v_new, rotary_positions, phases, axes,
                   block_tables, context_lens, interleaved=False)
    decode_shared_prefix(out, q, k_cache, v_cache, prefix_tables, prefix_lens, block_tables,
                         context_lens, scale, max_prefix_len, max_context_len, workspace=None)
    workspace_size_shared_prefix(q, k_cache, prefix_tables, block_tables, out_dtype,
                                 max_prefix_len, max_context_len)
    decode_accumulate(out, new_weights, q, k_cache, v_cache, block_tables, context_lens, scale,
                      max_context_len, weights=None, workspace=None)
    workspace_size_accumulate(q, k_cache, block_tables, out_dtype, max_context_len)
    evict_kv(k_cache, v_cache, weights, block_tables, context_lens, new_block_tables,
             new_weights, new_lens, kept, sink=0, recent=0)
    workspace_size(q, k_cache, block_tables, out_dtype, max_context_len, partition_tokens=0)
    workspace_size_multi(q, k_cache, block_tables, out_dtype, max_context_len, partition_tokens=0)
    plan_info(q, k_cache, block_tables, max_context_len, partition_tokens=0)
    choose_partition_tokens(q, k_cache, block_tables, max_context_len, num_sms)
    resolve_blocks(out_phys, block_tables, context_lens, block_size, num_blocks)
    selftest_wait_timeout(timeout_ns)
    device_error()
    set_switch(which, value) / get_switch(which)     (test and tuning switches)

Every launching call also takes ``stream=`` (default: the current torch stream).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

__all__ = ["PaError", "decode", "decode_splitkv", "decode_splitkv_noalloc", "decode_multi",
           "append_kv", "rope_phases", "rope_append_kv", "decode_shared_prefix",
           "workspace_size_shared_prefix", "decode_accumulate", "workspace_size_accumulate",
           "evict_kv", "workspace_size", "workspace_size_multi", "plan_info", "choose_partition_tokens",
           "resolve_blocks", "selftest_wait_timeout", "device_error", "library_path", "F16",
           "BF16", "F32", "PARTITION_BALANCED", "set_switch", "get_switch", "SWITCH_MULTI_KERNEL",
           "SWITCH_TILE_COMPACT_Q", "KERNEL_AUTO", "KERNEL_MMA", "KERNEL_TILE"]

F16, BF16, F32 = 0, 1, 2
PARTITION_BALANCED = -1   # partition_tokens value requesting the balanced split
SWITCH_MULTI_KERNEL, SWITCH_TILE_COMPACT_Q = 0, 1      # pa_set_switch switches
KERNEL_AUTO, KERNEL_MMA, KERNEL_TILE = 0, 1, 2         # values of SWITCH_MULTI_KERNEL
_STATUS = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_WORKSPACE",
           4: "PA_ERR_CUDA", 5: "PA_ERR_TIMEOUT"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libpa_decode.so")
_lock = threading.Lock()
_lib = None


class PaError(RuntimeError):
    """A non-OK pa_status returned by the library."""

    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_STATUS.get(code, code)}")


class _Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int64), ("kv_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with "
                    "`python -m paged_kv_attention_08_gb300.build` (there is no fallback path)")
            lib = ctypes.CDLL(_LIB_PATH)
            P, S = ctypes.c_void_p, ctypes.POINTER(_Shape)
            i32, f32, sz = ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
            lib.pa_decode.argtypes = [P, P, P, P, P, P, S, f32, P]
            lib.pa_decode.restype = ctypes.c_int
            lib.pa_decode_splitkv.argtypes = [P, P, P, P, P, P, S, f32, i32, i32, P, sz, P]
            lib.pa_decode_splitkv.restype = ctypes.c_int
            lib.pa_decode_splitkv_noalloc.argtypes = [P, P, P, P, P, P, S, f32, i32, i32, P]
            lib.pa_decode_splitkv_noalloc.restype = ctypes.c_int
            lib.pa_decode_multi.argtypes = [P, P, P, P, P, P, S, i32, f32, i32, i32, P, sz, P]
            lib.pa_decode_multi.restype = ctypes.c_int
            lib.pa_plan_info.argtypes = [S, i32, i32, i32, P]
            lib.pa_plan_info.restype = ctypes.c_int
            lib.pa_workspace_size_multi.argtypes = [S, i32, i32, i32]
            lib.pa_workspace_size_multi.restype = sz
            lib.pa_workspace_size.argtypes = [S, i32, i32]
            lib.pa_workspace_size.restype = sz
            lib.pa_choose_partition_tokens.argtypes = [S, i32, i32]
            lib.pa_choose_partition_tokens.restype = i32
            lib.pa_resolve_blocks.argtypes = [P, P, P, S, P]
            lib.pa_resolve_blocks.restype = ctypes.c_int
            lib.pa_append_kv.argtypes = [P, P, P, P, P, P, S, P]
            lib.pa_append_kv.restype = ctypes.c_int
            lib.pa_rope_append_kv.argtypes = [P] * 11 + [S, i32, ctypes.POINTER(_Rope), P]
            lib.pa_rope_append_kv.restype = ctypes.c_int
            lib.pa_decode_shared_prefix.argtypes = [P] * 8 + [S, i32, i32, i32, f32, i32, i32, P, sz, P]
            lib.pa_decode_shared_prefix.restype = ctypes.c_int
            lib.pa_workspace_size_shared_prefix.argtypes = [S, i32, i32, i32, i32, i32]
            lib.pa_workspace_size_shared_prefix.restype = sz
            lib.pa_decode_accumulate.argtypes = [P] * 8 + [S, i32, f32, i32, P, sz, P]
            lib.pa_decode_accumulate.restype = ctypes.c_int
            lib.pa_workspace_size_accumulate.argtypes = [S, i32, i32]
            lib.pa_workspace_size_accumulate.restype = sz
            lib.pa_evict_kv.argtypes = [P] * 9 + [S, i32, i32, i32, i32, P]
            lib.pa_evict_kv.restype = ctypes.c_int
            lib.pa_selftest_wait_timeout.argtypes = [ctypes.c_uint64, P]
            lib.pa_selftest_wait_timeout.restype = ctypes.c_int
            lib.pa_device_error.argtypes = [ctypes.POINTER(i32), P]
            lib.pa_device_error.restype = ctypes.c_int
            lib.pa_set_switch.argtypes = [i32, i32]
            lib.pa_set_switch.restype = ctypes.c_int
            lib.pa_get_switch.argtypes = [i32]
            lib.pa_get_switch.restype = i32
            lib.pa_status_string.argtypes = [ctypes.c_int]
            lib.pa_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float16:
        return F16
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {dt}")


def make_shape(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
               out_dtype: torch.dtype | None = None) -> _Shape:
    """pa_shape from tensor shapes: q [B,H,D], k_cache [NB,bs,Hkv,D], block_tables [B,max_blocks]."""
    if q.dim() != 3 or k_cache.dim() != 4 or block_tables.dim() != 2:
        raise ValueError("expected q [B,H,D], k_cache [NB,bs,Hkv,D], block_tables [B,max_blocks]")
    B, H, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    return _Shape(B, H, Hkv, D, bs, block_tables.shape[1], NB, _dtype_code(k_cache.dtype),
                  _dtype_code(out_dtype if out_dtype is not None else q.dtype))


def _stream_ptr(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(code: int, what: str):
    if code != 0:
        raise PaError(code, what)


def _dev_tensors(*ts):
    dev = None
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on one device")


def _ints(block_tables, context_lens):
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")


def _check_args(out, q, k_cache, v_cache, block_tables, context_lens, multi=False):
    """Shapes and dtypes that the library takes on trust: it reads the problem
    shape from q, k_cache and block_tables alone, so a v_cache, out, table or
    length tensor of another shape or dtype would be read or written past its
    memory.  Raises ValueError / TypeError before anything reaches the device."""
    if q.dim() != (4 if multi else 3):
        raise ValueError("q must be [batch, q_len, num_heads, head_dim]" if multi
                         else "q must be [batch, num_heads, head_dim]")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]")
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError(f"v_cache {tuple(v_cache.shape)} must be shaped like k_cache "
                         f"{tuple(k_cache.shape)}")
    if v_cache.dtype != k_cache.dtype:
        raise TypeError("v_cache must have k_cache's dtype")
    if q.dtype != k_cache.dtype:
        raise TypeError("q must have the cache's dtype")
    if q.shape[-1] != k_cache.shape[3]:
        raise ValueError(f"q's head_dim {q.shape[-1]} differs from the cache's {k_cache.shape[3]}")
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out {tuple(out.shape)} must be shaped like q {tuple(q.shape)}")
    if out.dtype not in (torch.float32, q.dtype):
        raise TypeError("out must be float32 or q's dtype")
    if block_tables.dim() != 2 or block_tables.shape[0] != q.shape[0]:
        raise ValueError("block_tables must be [batch, max_blocks_per_seq]")
    if context_lens.dim() != 1 or context_lens.numel() != q.shape[0]:
        raise ValueError("context_lens must be [batch]")
    _ints(block_tables, context_lens)


def decode(out, q, k_cache, v_cache, block_tables, context_lens, scale: float, stream=None):
    """Single-pass paged decode into ``out`` ([B,H,D], fp32 or q's dtype)."""
    _check_args(out, q, k_cache, v_cache, block_tables, context_lens)
    _dev_tensors(out, q, k_cache, v_cache, block_tables, context_lens)
    shape = make_shape(q, k_cache, block_tables, out.dtype)
    _check(_load().pa_decode(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             block_tables.data_ptr(), context_lens.data_ptr(),
                             ctypes.byref(shape), float(scale), _stream_ptr(stream)), "pa_decode")
    return out


def workspace_size(q, k_cache, block_tables, out_dtype, max_context_len: int,
                   partition_tokens: int = 0) -> int:
    shape = make_shape(q, k_cache, block_tables, out_dtype)
    return int(_load().pa_workspace_size(ctypes.byref(shape), int(max_context_len),
                                         int(partition_tokens)))


def choose_partition_tokens(q, k_cache, block_tables, max_context_len: int, num_sms: int) -> int:
    shape = make_shape(q, k_cache, block_tables, None)
    return int(_load().pa_choose_partition_tokens(ctypes.byref(shape), int(max_context_len),
                                                  int(num_sms)))


def decode_splitkv(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                   max_context_len: int, partition_tokens: int = 0, workspace=None, stream=None):
    """Flash-Decoding split-KV decode.  ``workspace`` is a CUDA byte tensor of at
    least ``workspace_size(...)`` bytes; when omitted one is taken from torch's
    allocator for this call."""
    _check_args(out, q, k_cache, v_cache, block_tables, context_lens)
    _dev_tensors(out, q, k_cache, v_cache, block_tables, context_lens)
    shape = make_shape(q, k_cache, block_tables, out.dtype)
    lib = _load()
    if workspace is None:
        need = lib.pa_workspace_size(ctypes.byref(shape), int(max_context_len), int(partition_tokens))
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=q.device)
    else:
        _dev_tensors(workspace)
    _check(lib.pa_decode_splitkv(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
                                 v_cache.data_ptr(), block_tables.data_ptr(),
                                 context_lens.data_ptr(), ctypes.byref(shape), float(scale),
                                 int(max_context_len), int(partition_tokens),
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream)), "pa_decode_splitkv")
    return out


def decode_splitkv_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                           max_context_len: int, partition_tokens: int = 0, stream=None):
    """Split-KV decode whose partials live in the library's fixed 16 MiB
    scratch instead of a caller workspace, for callers that cannot allocate
    device memory.  Calls that may overlap on the GPU race on that scratch;
    the first call on a device should come before any stream capture.
    Raises PaError (PA_ERR_WORKSPACE) when the partials would not fit."""
    _check_args(out, q, k_cache, v_cache, block_tables, context_lens)
    _dev_tensors(out, q, k_cache, v_cache, block_tables, context_lens)
    shape = make_shape(q, k_cache, block_tables, out.dtype)
    _check(_load().pa_decode_splitkv_noalloc(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(), ctypes.byref(shape), float(scale),
        int(max_context_len), int(partition_tokens), _stream_ptr(stream)),
        "pa_decode_splitkv_noalloc")
    return out


def _multi_shape(q, k_cache, block_tables, out_dtype):
    if q.dim() != 4:
        raise ValueError("q must be [batch, q_len, num_heads, head_dim]")
    return make_shape(q[:, 0], k_cache, block_tables, out_dtype), int(q.shape[1])


class _PlanDesc(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("partitions", ctypes.c_int32),
                ("partition_tokens", ctypes.c_int32), ("reduce", ctypes.c_int32),
                ("ctas", ctypes.c_int32), ("threads", ctypes.c_int32)]


_KERNELS = {0: "mma.sync m16n8k16", 1: "tcgen05 tile"}
_REDUCE = {0: "none", 1: "cluster DSMEM", 2: "workspace+combine kernel", 3: "balanced split"}


def plan_info(q, k_cache, block_tables, max_context_len: int, partition_tokens: int = 0,
              out_dtype=None) -> dict:
    """The plan a split-KV call with these arguments uses on the current device
    (q [B, H, D] for one query token, [B, Q, H, D] for several)."""
    if q.dim() == 4:
        shape, q_len = _multi_shape(q, k_cache, block_tables, out_dtype or torch.float32)
    else:
        shape, q_len = make_shape(q, k_cache, block_tables, out_dtype or torch.float32), 1
    d = _PlanDesc()
    _check(_load().pa_plan_info(ctypes.byref(shape), q_len, int(max_context_len),
                                int(partition_tokens), ctypes.byref(d)), "pa_plan_info")
    return {"kernel": _KERNELS[d.kernel], "partitions": d.partitions,
            "partition_tokens": d.partition_tokens, "reduce": _REDUCE[d.reduce],
            "ctas": d.ctas, "threads": d.threads}


def workspace_size_multi(q, k_cache, block_tables, out_dtype, max_context_len: int,
                         partition_tokens: int = 0) -> int:
    shape, q_len = _multi_shape(q, k_cache, block_tables, out_dtype)
    return int(_load().pa_workspace_size_multi(ctypes.byref(shape), q_len, int(max_context_len),
                                               int(partition_tokens)))


def decode_multi(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                 max_context_len: int, partition_tokens: int = 0, workspace=None, stream=None):
    """Several query tokens per sequence (q, out: [B, Q, H, D]); query token i
    of sequence b attends causally to the cached tokens t <= context_lens[b] - Q + i."""
    _check_args(out, q, k_cache, v_cache, block_tables, context_lens, multi=True)
    _dev_tensors(out, q, k_cache, v_cache, block_tables, context_lens)
    shape, q_len = _multi_shape(q, k_cache, block_tables, out.dtype)
    lib = _load()
    if workspace is None:
        need = lib.pa_workspace_size_multi(ctypes.byref(shape), q_len, int(max_context_len),
                                           int(partition_tokens))
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=q.device)
    else:
        _dev_tensors(workspace)
    _check(lib.pa_decode_multi(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
                               v_cache.data_ptr(), block_tables.data_ptr(),
                               context_lens.data_ptr(), ctypes.byref(shape), q_len, float(scale),
                               int(max_context_len), int(partition_tokens), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "pa_decode_multi")
    return out


def append_kv(k_cache, v_cache, k_new, v_new, block_tables, positions, stream=None):
    """Write each sequence's new token ([B, Hkv, D] k_new / v_new) into its
    cache slot at ``positions[b]``; negative positions and masked entries
    write nothing."""
    if k_cache.dim() != 4 or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, "
                         "num_kv_heads, head_dim]")
    if v_cache.dtype != k_cache.dtype or k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype:
        raise TypeError("new keys/values and both caches must have one dtype")
    if block_tables.dim() != 2 or positions.dim() != 1 or positions.numel() != block_tables.shape[0]:
        raise ValueError("block_tables must be [batch, max_blocks_per_seq], positions [batch]")
    _ints(block_tables, positions)
    B = block_tables.shape[0]
    NB, bs, Hkv, D = k_cache.shape
    if tuple(k_new.shape) != (B, Hkv, D) or tuple(v_new.shape) != (B, Hkv, D):
        raise ValueError("k_new/v_new must be [batch, num_kv_heads, head_dim]")
    _dev_tensors(k_cache, v_cache, k_new, v_new, block_tables, positions)
    shape = _Shape(B, Hkv, Hkv, D, bs, block_tables.shape[1], NB, _dtype_code(k_cache.dtype), F32)
    _check(_load().pa_append_kv(k_cache.data_ptr(), v_cache.data_ptr(), k_new.data_ptr(),
                                v_new.data_ptr(), block_tables.data_ptr(), positions.data_ptr(),
                                ctypes.byref(shape), _stream_ptr(stream)), "pa_append_kv")


# The serving-step entry points below run once per layer and step, where the
# binding's own time shows: they check with as few calls as that takes, and
# launch on the tensors' device whatever the current one is.

def _device_of(t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    return dev


def _same_device(dev: int, ts, contiguous: bool = True):
    for t in ts:
        if t.get_device() != dev:
            raise ValueError("all tensors must be CUDA tensors on one device")
        if contiguous and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _stream_on(dev: int, stream) -> int:
    """The given stream, or the device's current one, for the C ABI."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError("stream is on another device than the tensors")
    return stream.cuda_stream


_KV_CODE = {torch.float16: F16, torch.bfloat16: BF16}


_2_31 = 1 << 31


def _i32(x, name) -> int:
    """A whole number of any kind (numpy's, a tensor's) as the C ABI's int32.
    (The calls of a step test for a plain one themselves.)"""
    x = int(x)
    if not -_2_31 <= x < _2_31:
        raise ValueError(f"{name} {x} does not fit in 32 bits")
    return x


def _attention_shape(out, q, k_cache, v_cache, block_tables, context_lens):
    """Checks what ``_check_args`` checks; pa_shape and q_len of a one-token
    ([B, H, D]) or several-token ([B, Q, H, D]) query."""
    qs, ks, bts = q.shape, k_cache.shape, block_tables.shape
    if len(qs) == 3:
        B, H, D = qs
        Q = 1
    elif len(qs) == 4:
        B, Q, H, D = qs
        if Q < 1:
            raise ValueError("q_len must be at least 1")
    else:
        raise ValueError("q must be [batch, num_heads, head_dim] or "
                         "[batch, q_len, num_heads, head_dim]")
    if len(ks) != 4 or v_cache.shape != ks:
        raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, "
                         "num_kv_heads, head_dim]")
    dt, odt = k_cache.dtype, out.dtype
    if q.dtype != dt or v_cache.dtype != dt:
        raise TypeError("q and both caches must have one dtype")
    if dt not in _KV_CODE:
        raise TypeError(f"unsupported dtype {dt}")
    if D != ks[3]:
        raise ValueError(f"q's head_dim {D} differs from the cache's {ks[3]}")
    if out.shape != qs:
        raise ValueError(f"out {tuple(out.shape)} must be shaped like q {tuple(qs)}")
    if odt != dt and odt != torch.float32:
        raise TypeError("out must be float32 or q's dtype")
    if len(bts) != 2 or bts[0] != B:
        raise ValueError("block_tables must be [batch, max_blocks_per_seq]")
    if context_lens.shape != (B,):
        raise ValueError("context_lens must be [batch]")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    code = _KV_CODE[dt]
    return _Shape(B, H, ks[2], D, ks[1], bts[1], ks[0], code, code if odt == dt else F32), Q


def _workspace_for(workspace, need, dev: int, stream):
    """The caller's workspace, or one from torch's allocator: (tensor, bytes).
    One taken here belongs to the stream that the call launches on."""
    if workspace is None:
        if need > 1 << 62:
            raise PaError(3, "workspace")
        with torch.cuda.stream(stream):  # (None: the current stream)
            workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=f"cuda:{dev}")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the tensors' device")
    return workspace, workspace.numel() * workspace.element_size()


def rope_phases(inv_freq: torch.Tensor) -> torch.Tensor:
    """The int64 table that ``rope_append_kv`` takes for the rotary frequencies
    ``inv_freq`` (float64, radians per position, one per pair; 1-D): each as a
    fraction of a turn, times 2^64.  Made once, kept by the caller."""
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise TypeError("inv_freq must be a 1-D float64 tensor")
    if not bool(torch.isfinite(inv_freq).all()):
        raise ValueError("inv_freq must be finite")
    turns = inv_freq / (2 * math.pi)
    turns = turns - torch.floor(turns + 0.5)  # in [-1/2, 1/2)
    return (turns * 2.0 ** 64).to(torch.int64)


def _token_stride(t, name, shape):
    """Elements between consecutive tokens of a [batch, q_len, heads, head_dim]
    view whose tokens lie evenly apart and whose rows are contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name} {tuple(t.shape)} must be {tuple(shape)}")
    batch, q_len, heads, head_dim = shape
    sb, sq, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != head_dim):
        raise ValueError(f"{name}'s heads must be contiguous")
    if q_len == 1:
        return sb if batch > 1 else heads * head_dim
    if batch > 1 and sb != q_len * sq:
        raise ValueError(f"{name}'s tokens must lie evenly apart")
    return sq


def rope_append_kv(q_out, k_cache, v_cache, q, k_new, v_new, rotary_positions, phases, axes,
                   block_tables, context_lens, interleaved: bool = False, stream=None):
    """Turn the new tokens' queries into ``q_out`` (``q`` itself, or memory of
    its own) and write their turned keys and their values into the paged cache.

    q, q_out [B, Q, H, D]; k_new, v_new [B, Q, Hkv, D] (views of one fused
    projection are fine); rotary_positions int32 [axes, B, Q]; phases from
    ``rope_phases`` and axes int32, one per rotary pair (2 * pairs <= D).
    context_lens counts the Q new tokens.  For one token per sequence the
    tensors may leave out their Q dimension."""
    if q.dim() == 3:
        if q_out.dim() != 3 or k_new.dim() != 3 or v_new.dim() != 3 or rotary_positions.dim() != 2:
            raise ValueError("q, q_out, k_new, v_new and rotary_positions must all leave out "
                             "the query-token dimension, or none")
        rope_append_kv(q_out.unsqueeze(1), k_cache, v_cache, q.unsqueeze(1), k_new.unsqueeze(1),
                       v_new.unsqueeze(1), rotary_positions.unsqueeze(2), phases, axes,
                       block_tables, context_lens, interleaved, stream)
        return q_out
    qs, ks, bts, rs = q.shape, k_cache.shape, block_tables.shape, rotary_positions.shape
    if len(qs) != 4:
        raise ValueError("q must be [batch, q_len, num_heads, head_dim]")
    if len(ks) != 4 or v_cache.shape != ks:
        raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, "
                         "num_kv_heads, head_dim]")
    dt = k_cache.dtype
    if v_cache.dtype != dt or q.dtype != dt or q_out.dtype != dt or k_new.dtype != dt or \
            v_new.dtype != dt:
        raise TypeError("queries, new keys/values and both caches must have one dtype")
    if dt not in _KV_CODE:
        raise TypeError(f"unsupported dtype {dt}")
    B, Q, H, D = qs
    NB, bs, Hkv, cache_d = ks
    if cache_d != D:
        raise ValueError(f"q's head_dim {D} differs from the cache's {cache_d}")
    if Q < 1:
        raise ValueError("q_len must be at least 1")
    if len(rs) != 3 or rs[1] != B or rs[2] != Q:
        raise ValueError("rotary_positions must be [axes, batch, q_len]")
    pairs = phases.numel()
    if rotary_positions.dtype != torch.int32 or axes.dtype != torch.int32:
        raise TypeError("rotary_positions and axes must be int32")
    if phases.dtype != torch.int64:
        raise TypeError("phases must be the int64 table of rope_phases")
    if phases.dim() != 1 or axes.shape != (pairs,):
        raise ValueError("phases and axes must hold one value per rotary pair")
    if len(bts) != 2 or bts[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [batch, max_blocks_per_seq], context_lens [batch]")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    rope = _Rope(2 * pairs, rs[0], 1 if interleaved else 0, 0,
                 _token_stride(q, "q", qs), _token_stride(q_out, "q_out", qs),
                 _token_stride(k_new, "k_new", (B, Q, Hkv, D)),
                 _token_stride(v_new, "v_new", (B, Q, Hkv, D)))
    dev = _device_of(k_cache)
    _same_device(dev, (k_cache, v_cache, rotary_positions, phases, axes, block_tables, context_lens))
    _same_device(dev, (q, q_out, k_new, v_new), contiguous=False)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return rope_append_kv(q_out, k_cache, v_cache, q, k_new, v_new, rotary_positions,
                                  phases, axes, block_tables, context_lens, interleaved, stream)
    _check((_lib or _load()).pa_rope_append_kv(
        q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), q.data_ptr(), k_new.data_ptr(),
        v_new.data_ptr(), rotary_positions.data_ptr(), phases.data_ptr(), axes.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(),
        _Shape(B, H, Hkv, D, bs, bts[1], NB, _KV_CODE[dt], F32), Q, rope,
        _stream_on(dev, stream)), "pa_rope_append_kv")
    return q_out


def _sizing_shape(q, k_cache, block_tables, out_dtype):
    """pa_shape, q_len and device for a workspace query."""
    if q.dim() == 4:
        shape, q_len = _multi_shape(q, k_cache, block_tables, out_dtype)
    else:
        shape, q_len = make_shape(q, k_cache, block_tables, out_dtype), 1
    return shape, q_len, _device_of(k_cache)


def _check_prefixes(prefix_tables, batch):
    shape = prefix_tables.shape
    if len(shape) != 2 or shape[0] < 1 or batch % shape[0]:
        raise ValueError("prefix_tables must be [prefixes, max_prefix_blocks], with as many "
                         "sequences for each prefix")
    if prefix_tables.dtype != torch.int32:
        raise TypeError("prefix_tables must be int32")
    return shape


def workspace_size_shared_prefix(q, k_cache, prefix_tables, block_tables, out_dtype,
                                 max_prefix_len: int, max_context_len: int) -> int:
    """Bytes of workspace that ``decode_shared_prefix`` takes, on the tensors' device."""
    shape, q_len, dev = _sizing_shape(q, k_cache, block_tables, out_dtype)
    P, mpb = _check_prefixes(prefix_tables, shape.batch)
    with torch.cuda.device(dev):
        return int(_load().pa_workspace_size_shared_prefix(
            shape, P, mpb, q_len, _i32(max_prefix_len, "max_prefix_len"),
            _i32(max_context_len, "max_context_len")))


def decode_shared_prefix(out, q, k_cache, v_cache, prefix_tables, prefix_lens, block_tables,
                         context_lens, scale: float, max_prefix_len: int, max_context_len: int,
                         workspace=None, stream=None):
    """Attention of a batch over shared prefixes and each sequence's own pages,
    as over one sequence.  q, out [B, H, D] or [B, Q, H, D]; prefix_tables int32
    [P, max_prefix_blocks] and prefix_lens int32 [P], sequence b having prefix
    b // (B // P); block_tables and context_lens are the sequences' own (the
    lengths count the Q new tokens, causal among themselves).  ``workspace``: a
    CUDA byte tensor of ``workspace_size_shared_prefix(...)`` bytes, else one
    is taken from torch's allocator."""
    shape, q_len = _attention_shape(out, q, k_cache, v_cache, block_tables, context_lens)
    P, mpb = _check_prefixes(prefix_tables, shape.batch)
    if prefix_lens.shape != (P,):
        raise ValueError("prefix_lens must be [prefixes]")
    if prefix_lens.dtype != torch.int32:
        raise TypeError("prefix_lens must be int32")
    if type(max_prefix_len) is not int or not -_2_31 <= max_prefix_len < _2_31:
        max_prefix_len = _i32(max_prefix_len, "max_prefix_len")
    if type(max_context_len) is not int or not -_2_31 <= max_context_len < _2_31:
        max_context_len = _i32(max_context_len, "max_context_len")
    if type(scale) is not float:
        scale = float(scale)
    dev = _device_of(k_cache)
    _same_device(dev, (out, q, k_cache, v_cache, prefix_tables, prefix_lens, block_tables,
                       context_lens))
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return decode_shared_prefix(out, q, k_cache, v_cache, prefix_tables, prefix_lens,
                                        block_tables, context_lens, scale, max_prefix_len,
                                        max_context_len, workspace, stream)
    lib = _lib or _load()
    need = 0 if workspace is not None else lib.pa_workspace_size_shared_prefix(
        shape, P, mpb, q_len, max_prefix_len, max_context_len)
    ws, ws_bytes = _workspace_for(workspace, need, dev, stream)
    _check(lib.pa_decode_shared_prefix(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        prefix_tables.data_ptr(), prefix_lens.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), shape, P, mpb, q_len, scale, max_prefix_len, max_context_len,
        ws.data_ptr(), ws_bytes, _stream_on(dev, stream)), "pa_decode_shared_prefix")
    return out


def workspace_size_accumulate(q, k_cache, block_tables, out_dtype, max_context_len: int) -> int:
    """Bytes of workspace that ``decode_accumulate`` takes, on the tensors' device."""
    shape, q_len, dev = _sizing_shape(q, k_cache, block_tables, out_dtype)
    with torch.cuda.device(dev):
        return int(_load().pa_workspace_size_accumulate(
            shape, q_len, _i32(max_context_len, "max_context_len")))


def decode_accumulate(out, new_weights, q, k_cache, v_cache, block_tables, context_lens,
                      scale: float, max_context_len: int, weights=None, workspace=None,
                      stream=None):
    """``decode_splitkv`` (q [B, H, D]) or ``decode_multi`` (q [B, Q, H, D]) that also
    adds every cached token's attention weight, summed over the kv head's
    query heads and the query tokens: new_weights[b, kvh, t] = weights[b, kvh, t] +
    sum p (fp32 [B, Hkv, max_blocks * block_size]; ``weights`` omitted: in place).
    Entries past a sequence's tokens are not written."""
    weights = new_weights if weights is None else weights
    shape, q_len = _attention_shape(out, q, k_cache, v_cache, block_tables, context_lens)
    want = (shape.batch, shape.num_kv_heads, shape.max_blocks_per_seq * shape.block_size)
    if weights.shape != want or new_weights.shape != want:
        raise ValueError(f"weights and new_weights must be {want}")
    if weights.dtype != torch.float32 or new_weights.dtype != torch.float32:
        raise TypeError("weights and new_weights must be float32")
    if type(max_context_len) is not int or not -_2_31 <= max_context_len < _2_31:
        max_context_len = _i32(max_context_len, "max_context_len")
    if type(scale) is not float:
        scale = float(scale)
    dev = _device_of(k_cache)
    _same_device(dev, (out, q, k_cache, v_cache, block_tables, context_lens, weights, new_weights))
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return decode_accumulate(out, new_weights, q, k_cache, v_cache, block_tables,
                                     context_lens, scale, max_context_len, weights, workspace,
                                     stream)
    lib = _lib or _load()
    need = 0 if workspace is not None else lib.pa_workspace_size_accumulate(
        shape, q_len, max_context_len)
    ws, ws_bytes = _workspace_for(workspace, need, dev, stream)
    _check(lib.pa_decode_accumulate(
        out.data_ptr(), new_weights.data_ptr(), weights.data_ptr(), q.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
        shape, q_len, scale, max_context_len, ws.data_ptr(), ws_bytes, _stream_on(dev, stream)),
        "pa_decode_accumulate")
    return out


def evict_kv(k_cache, v_cache, weights, block_tables, context_lens, new_block_tables, new_weights,
             new_lens, kept, sink: int = 0, recent: int = 0, stream=None):
    """Cut every kv head of every sequence down to ``kept.shape[2]`` tokens: the
    first ``sink`` and last ``recent`` ones and those of the largest
    accumulated ``weights`` ([B, Hkv, max_blocks * block_size] fp32, ties to
    the lowest index), moved in their order to the front of
    ``new_block_tables``' pages.  Passing ``block_tables`` / ``weights``
    themselves as the new ones works in place (and so, more slowly, does a copy
    of ``block_tables`` or of its first columns); other tables must hold other
    pages than any sequence's old ones.  ``kept`` (int32 [B, Hkv,
    budget]) receives the kept tokens' former positions, ``new_lens`` (int32
    [B]) the new lengths."""
    ks, bts, nbts, kts = k_cache.shape, block_tables.shape, new_block_tables.shape, kept.shape
    if len(ks) != 4 or v_cache.shape != ks:
        raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, "
                         "num_kv_heads, head_dim]")
    dt = k_cache.dtype
    if v_cache.dtype != dt:
        raise TypeError("v_cache must have k_cache's dtype")
    if dt not in _KV_CODE:
        raise TypeError(f"unsupported dtype {dt}")
    if len(bts) != 2 or len(nbts) != 2 or nbts[0] != bts[0]:
        raise ValueError("block_tables and new_block_tables must be [batch, max_blocks_per_seq]")
    NB, bs, Hkv, D = ks
    B, mb = bts
    new_mb = nbts[1]
    if weights.shape != (B, Hkv, mb * bs) or new_weights.shape != (B, Hkv, new_mb * bs):
        raise ValueError("weights and new_weights must be [batch, num_kv_heads, their table's "
                         "max_blocks * block_size]")
    if weights.dtype != torch.float32 or new_weights.dtype != torch.float32:
        raise TypeError("weights and new_weights must be float32")
    if context_lens.shape != (B,) or new_lens.shape != (B,):
        raise ValueError("context_lens and new_lens must be [batch]")
    if len(kts) != 3 or kts[0] != B or kts[1] != Hkv:
        raise ValueError("kept must be [batch, num_kv_heads, budget]")
    i32 = torch.int32
    if block_tables.dtype != i32 or context_lens.dtype != i32 or new_block_tables.dtype != i32 or \
            new_lens.dtype != i32 or kept.dtype != i32:
        raise TypeError("block tables, lengths and kept must be int32")
    if type(sink) is not int or not -_2_31 <= sink < _2_31:
        sink = _i32(sink, "sink")
    if type(recent) is not int or not -_2_31 <= recent < _2_31:
        recent = _i32(recent, "recent")
    dev = _device_of(k_cache)
    _same_device(dev, (k_cache, v_cache, weights, block_tables, context_lens, new_block_tables,
                       new_weights, new_lens, kept))
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return evict_kv(k_cache, v_cache, weights, block_tables, context_lens,
                            new_block_tables, new_weights, new_lens, kept, sink, recent, stream)
    _check((_lib or _load()).pa_evict_kv(
        k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), new_block_tables.data_ptr(), new_weights.data_ptr(),
        new_lens.data_ptr(), kept.data_ptr(),
        _Shape(B, Hkv, Hkv, D, bs, mb, NB, _KV_CODE[dt], F32), new_mb, kts[2], sink, recent,
        _stream_on(dev, stream)), "pa_evict_kv")
    return new_lens


def resolve_blocks(out_phys, block_tables, context_lens, block_size: int, num_blocks: int,
                   stream=None):
    """Physical block the kernels read for each (sequence, logical page); -1 if none."""
    if out_phys.dtype != torch.int32 or out_phys.shape != block_tables.shape:
        raise ValueError("out_phys must be int32 shaped like block_tables")
    if block_tables.dim() != 2 or context_lens.dim() != 1 or \
            context_lens.numel() != block_tables.shape[0]:
        raise ValueError("block_tables must be [batch, max_blocks_per_seq], context_lens [batch]")
    _ints(block_tables, context_lens)
    _dev_tensors(out_phys, block_tables, context_lens)
    B, mb = block_tables.shape
    shape = _Shape(B, 1, 1, 64, int(block_size), mb, int(num_blocks), F16, F32)
    _check(_load().pa_resolve_blocks(out_phys.data_ptr(), block_tables.data_ptr(),
                                     context_lens.data_ptr(), ctypes.byref(shape),
                                     _stream_ptr(stream)), "pa_resolve_blocks")
    return out_phys


def selftest_wait_timeout(timeout_ns: int, stream=None):
    """Run the bounded-wait self-test kernel (it records PA_ERR_TIMEOUT)."""
    _check(_load().pa_selftest_wait_timeout(int(timeout_ns), _stream_ptr(stream)),
           "pa_selftest_wait_timeout")


def device_error(stream=None) -> int:
    """Read and clear the device error word (synchronises the stream)."""
    code = ctypes.c_int32(0)
    _check(_load().pa_device_error(ctypes.byref(code), _stream_ptr(stream)), "pa_device_error")
    return int(code.value)


def set_switch(which: int, value: int):
    """Set a test / tuning switch (SWITCH_MULTI_KERNEL: KERNEL_AUTO, KERNEL_MMA or
    KERNEL_TILE; SWITCH_TILE_COMPACT_Q: 1 or 0) for every later call."""
    _check(_load().pa_set_switch(int(which), int(value)), "pa_set_switch")


def get_switch(which: int) -> int:
    return int(_load().pa_get_switch(int(which)))
