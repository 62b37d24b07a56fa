"""ctypes binding of ``libpagedkv.so`` (``include/pagedkv.h``).

Argument marshalling only: tensors become device pointers, the cache tensor's
shape becomes a ``pkv_cache_desc``, and the current PyTorch stream becomes the
``stream`` argument.  Every step of the path runs in the library's kernels.
The library must have been built (``paged_kv_cache_11_gb300._build``); there is
no fallback of any kind.
"""
from __future__ import annotations

import array
import ctypes
import operator
from pathlib import Path
from typing import Sequence

import torch

LIB_PATH = Path(__file__).resolve().parent / "_lib" / "libpagedkv.so"

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA, PKV_ERR_DEVICE_METADATA = range(6)
PKV_BF16, PKV_FP16, PKV_FP32, PKV_E4M3 = 0, 1, 2, 3
DEVERR_NAMES = {0: "none", 1: "slot", 2: "copy_id", 3: "context_len", 4: "block_id", 5: "timeout",
                6: "prefix_len", 7: "group", 8: "position", 9: "scale"}

_DTYPE_CODE = {torch.bfloat16: PKV_BF16, torch.float16: PKV_FP16, torch.float32: PKV_FP32,
               torch.float8_e4m3fn: PKV_E4M3}


class CacheDesc(ctypes.Structure):
    _fields_ = [
        ("num_blocks", ctypes.c_int64),
        ("num_kv_heads", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class RopeDesc(ctypes.Structure):
    _fields_ = [
        ("num_q_heads", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("max_position", ctypes.c_int64),
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("norm_eps", ctypes.c_float),
    ]


class PagedKVError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_LIB: ctypes.CDLL | None = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is not None:
        return _LIB
    if not LIB_PATH.exists():
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m paged_kv_cache_11_gb300._build` "
            "(or __graft_entry__.build()) first")
    lib = ctypes.CDLL(str(LIB_PATH))
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    desc_p = ctypes.POINTER(CacheDesc)
    lib.pkv_status_string.argtypes = [ctypes.c_int]
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_version.argtypes = []
    lib.pkv_version.restype = ctypes.c_int
    lib.pkv_launch_count.argtypes = []
    lib.pkv_launch_count.restype = ctypes.c_uint64
    lib.paged_kv_append.argtypes = [vp, vp, vp, i64, vp, vp, desc_p, vp]
    lib.paged_kv_append.restype = ctypes.c_int
    rope_p = ctypes.POINTER(RopeDesc)
    lib.paged_kv_append_rope.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, desc_p, rope_p, vp]
    lib.paged_kv_append_rope.restype = ctypes.c_int
    lib.paged_kv_append_rope_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, desc_p, rope_p,
                                             vp]
    lib.paged_kv_append_rope_fp8.restype = ctypes.c_int
    lib.paged_attention_decode_fp8.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, ctypes.c_float,
                                               vp, i32, desc_p, i32, vp, sz, vp]
    lib.paged_attention_decode_fp8.restype = ctypes.c_int
    lib.copy_blocks_fp8.argtypes = [vp, vp, vp, vp, i32, vp, i32, desc_p, vp]
    lib.copy_blocks_fp8.restype = ctypes.c_int
    lib.paged_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.paged_attention_workspace_bytes.restype = sz
    lib.paged_attention_plan.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.paged_attention_plan.restype = i32
    lib.paged_attention_partition_size.argtypes = [i32, i32, i32, i32, i32]
    lib.paged_attention_partition_size.restype = i32
    lib.paged_attention_decode.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, ctypes.c_float, vp, i32,
                                           desc_p, i32, vp, sz, vp]
    lib.paged_attention_decode.restype = ctypes.c_int
    lib.paged_attention_append_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32,
                                                  ctypes.c_float, vp, i32, desc_p, i32, vp, sz, vp]
    lib.paged_attention_append_decode.restype = ctypes.c_int
    lib.paged_attention_decode_static.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, ctypes.c_float, vp,
                                                  i32, desc_p, i32, vp]
    lib.paged_attention_decode_static.restype = ctypes.c_int
    lib.paged_attention_decode_grouped.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, i32, i32, vp, i32,
                                                   ctypes.c_float, vp, i32, desc_p, i32, vp, sz, vp]
    lib.paged_attention_decode_grouped.restype = ctypes.c_int
    lib.paged_attention_append_decode_grouped.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, i32,
                                                          i32, vp, i32, ctypes.c_float, vp, i32, desc_p, i32, vp, sz,
                                                          vp]
    lib.paged_attention_append_decode_grouped.restype = ctypes.c_int
    lib.paged_attention_grouped_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.paged_attention_grouped_workspace_bytes.restype = sz
    lib.copy_blocks.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), i32, vp, i32, desc_p, vp]
    lib.copy_blocks.restype = ctypes.c_int
    lib.swap_blocks.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), i64, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                i64, i32, vp, i32, desc_p, vp]
    lib.swap_blocks.restype = ctypes.c_int
    lib.compact_tokens.argtypes = [vp, vp, i64, vp, vp, desc_p, vp]
    lib.compact_tokens.restype = ctypes.c_int
    lib.pkv_check_device_error.argtypes = [vp, ctypes.POINTER(i32)]
    lib.pkv_check_device_error.restype = ctypes.c_int
    lib.pkv_wait_selftest.argtypes = [i32, vp]
    lib.pkv_wait_selftest.restype = ctypes.c_int
    _LIB = lib
    return lib


def status_string(status: int) -> str:
    return _lib().pkv_status_string(int(status)).decode()


def version() -> int:
    return int(_lib().pkv_version())


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(_lib().pkv_launch_count())


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    """Descriptor of a cache tensor shaped [num_blocks, num_kv_heads, block_size, head_dim]."""
    if k_cache.dim() != 4:
        raise ValueError("cache must be [num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = k_cache.shape
    return CacheDesc(nb, hkv, bs, d, _DTYPE_CODE.get(k_cache.dtype, -1))


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _check(status: int, what: str) -> None:
    if status != PKV_OK:
        raise PagedKVError(status, what)


def paged_kv_append(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, stream=None) -> None:
    """Block write: k_cache[slot // bs, h, slot % bs] = k[t, h] for every token t (same for v)."""
    for t in (k, v, slot_mapping, k_cache, v_cache):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    _require(slot_mapping.dtype == torch.int64, "slot_mapping must be int64")
    desc = cache_desc(k_cache)
    _check(_lib().paged_kv_append(_ptr(k), _ptr(v), _ptr(slot_mapping), slot_mapping.numel(), _ptr(k_cache),
                                  _ptr(v_cache), ctypes.byref(desc), _stream(stream)), "paged_kv_append")


# A step's calls are short against the GPU's work: the checks below read each property of a tensor once.
_get_device, _is_contiguous, _numel = torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.numel
_dtype_of = operator.attrgetter("dtype")
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _one_device(tensors) -> int:
    """The index of the CUDA device that all the tensors are on, each of them contiguous."""
    devs = set(map(_get_device, tensors))
    dev = devs.pop()
    if devs or dev < 0:
        raise ValueError("tensors must be on one CUDA device")
    if not all(map(_is_contiguous, tensors)):
        raise ValueError("tensors must be contiguous")
    return dev


def _context(dev: int, stream):
    """What a call runs in where its device is not the current one or a stream is given: the device is current, and
    the call's allocations belong to the stream it launches on, so that none is handed out again while it still runs."""
    if stream is None:
        return torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    _require(stream.device.index == dev, "stream belongs to another device")
    return torch.cuda.stream(stream)


def _token_stride(t: torch.Tensor, want: tuple, dtype, dev: int) -> int:
    """Elements from one token's row to the next of q, k or v, shaped ``want`` = (tokens, heads, head_dim)."""
    if t.shape != want or t.dtype != dtype or t.get_device() != dev:
        raise ValueError("q is [num_tokens, num_q_heads, head_dim], k and v [num_tokens, num_kv_heads, head_dim], "
                         "of one dtype, on the caches' device")
    s0, s1, s2 = t.stride()
    n, heads, d = want
    if (s2 != 1 and d != 1) or (s1 != d and heads != 1):
        raise ValueError("a token's heads must be contiguous in q, k and v")
    return s0 if n > 1 else heads * d


def _append_rope(fn, name, q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, scales, q_norm, k_norm, norm_eps,
                 interleaved, q_out, stream):
    rest = [k_cache, v_cache, slot_mapping, *scales]
    rest += [t for t in (positions, cos_sin, q_norm, k_norm, q_out) if t is not None]
    dev = _one_device(rest)
    if stream is not None or _current_device() != dev:
        with _context(dev, stream):
            return _append_rope(fn, name, q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, scales, q_norm,
                                k_norm, norm_eps, interleaved, q_out, None)
    shape, dt, cache_dt = k_cache.shape, k.dtype, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != cache_dt:
        raise ValueError("caches must be [num_blocks, num_kv_heads, block_size, head_dim], K as V")
    nb, hkv, bs, d = shape
    if slot_mapping.dtype != _I64 or slot_mapping.dim() != 1:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    n = slot_mapping.numel()
    k_stride, v_stride = _token_stride(k, (n, hkv, d), dt, dev), _token_stride(v, (n, hkv, d), dt, dev)
    hq = q_stride = q_ptr = 0
    if q is not None:
        hq, q_ptr = q.shape[1] if q.dim() == 3 else -1, q.data_ptr()
        q_stride = _token_stride(q, (n, hq, d), dt, dev)
        if q_out is not None and (q_out.shape != q.shape or q_out.dtype != dt):
            raise ValueError("q_out is as q")
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm belong to q")
    rot = max_position = 0
    if cos_sin is not None:
        if positions is None or positions.dtype != _I64 or positions.dim() != 1 or positions.numel() != n:
            raise ValueError("positions must be int64 [num_tokens] where there is a cos_sin")
        if cos_sin.dtype != _F32 or cos_sin.dim() != 2 or cos_sin.shape[1] == 0:
            raise ValueError("cos_sin must be fp32 [max_position, rot_dim] (None: no rotation)")
        max_position, rot = cos_sin.shape
    elif positions is not None:
        raise ValueError("positions without cos_sin")
    for w in (q_norm, k_norm):
        if w is not None and (w.dtype != dt or w.shape != (d,)):
            raise ValueError("norm weights are [head_dim], of k's dtype")
    for s in scales:
        if s.dtype != _F32 or s.shape != (nb, hkv):
            raise ValueError("scales must be fp32 [num_blocks, num_kv_heads]")
    desc = CacheDesc(nb, hkv, bs, d, _DTYPE_CODE.get(cache_dt, -1))
    rope = RopeDesc(hq, _DTYPE_CODE.get(dt, -1), q_stride, k_stride, v_stride, max_position, rot, bool(interleaved),
                    float(norm_eps))

    if q_out is None and q is not None:
        q_out = torch.empty(q.shape, dtype=dt, device=q.device)
    st = fn(q_ptr, k.data_ptr(), v.data_ptr(), _ptr(positions), _ptr(cos_sin), _ptr(q_norm), _ptr(k_norm),
            slot_mapping.data_ptr(), n, _ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(),
            *[s.data_ptr() for s in scales], desc, rope, _raw_stream(dev))
    if st != PKV_OK:
        raise PagedKVError(st, name)
    return q_out


def paged_kv_append_rope(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None,
                         cos_sin: torch.Tensor | None, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, q_norm: torch.Tensor | None = None,
                         k_norm: torch.Tensor | None = None, norm_eps: float = 1e-6, interleaved: bool = False,
                         q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Block write with the rotation by position (and the RMS norm of each query and key head, where weights are
    given) on the way; returns ``q_out``, the rotated queries.

    q [num_tokens, num_q_heads, 128] (or None), k and v [num_tokens, num_kv_heads, 128] may be slices of one fused
    projection: only a token's heads must be contiguous.  ``cos_sin`` is fp32 [max_position, rot_dim], the cosines of
    a position's rot_dim / 2 angles before their sines (None: no rotation).  Rows of padding tokens (negative slots)
    are left as they were; ``q_out`` may be ``q`` where that is contiguous.
    """
    return _append_rope(_lib().paged_kv_append_rope, "paged_kv_append_rope", q, k, v, positions, cos_sin, slot_mapping,
                        k_cache, v_cache, (), q_norm, k_norm, norm_eps, interleaved, q_out, stream)


def paged_kv_append_rope_fp8(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None,
                             cos_sin: torch.Tensor | None, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                             q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None,
                             norm_eps: float = 1e-6, interleaved: bool = False, q_out: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor | None:
    """paged_kv_append_rope into float8_e4m3fn caches with one fp32 scale per (block, KV head), ``k_scales`` and
    ``v_scales`` [num_blocks, num_kv_heads]: a stored value stands for value * scale.

    A block starts afresh when its first row is written, and its scales follow the rows it takes on (the header has
    the rule); a block's tokens stand together in ``slot_mapping``.
    """
    return _append_rope(_lib().paged_kv_append_rope_fp8, "paged_kv_append_rope_fp8", q, k, v, positions, cos_sin,
                        slot_mapping, k_cache, v_cache, (k_scales, v_scales), q_norm, k_norm, norm_eps, interleaved,
                        q_out, stream)


def paged_attention_workspace_bytes(num_seqs: int, num_q_heads: int, head_dim: int, max_context_len: int,
                                    partition_size: int = 0) -> int:
    return int(_lib().paged_attention_workspace_bytes(num_seqs, num_q_heads, head_dim, max_context_len,
                                                      partition_size))


PLAN_NAMES = {0: "single", 1: "split", 2: "split+reduce"}


def paged_attention_plan(num_seqs: int, num_q_heads: int, num_kv_heads: int, block_size: int, max_context_len: int,
                         partition_size: int = 0) -> str:
    """Decomposition a decode call with these sizes uses on the current device."""
    k = int(_lib().paged_attention_plan(num_seqs, num_q_heads, num_kv_heads, block_size, max_context_len,
                                        partition_size))
    return PLAN_NAMES.get(k, "invalid")


def paged_attention_partition_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, max_context_len: int,
                                   partition_size: int = 0) -> int:
    """Split-K partition (tokens) a decode call with these sizes uses on the current device."""
    return int(_lib().paged_attention_partition_size(num_seqs, num_q_heads, num_kv_heads, max_context_len,
                                                     partition_size))


def paged_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                           out: torch.Tensor | None = None, max_context_len: int | None = None,
                           partition_size: int = 0, workspace: torch.Tensor | None = None,
                           out_dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """Paged decode attention; returns ``out`` [num_seqs, num_q_heads, head_dim].

    ``max_context_len`` bounds ``context_lens`` (default: the block tables'
    capacity).  A workspace is allocated with torch when one is needed and
    none is given.
    """
    for t in (q, k_cache, v_cache, block_tables, context_lens):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    _require(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32,
             "block_tables and context_lens must be int32")
    _require(q.dim() == 3 and block_tables.dim() == 2, "q is [num_seqs, num_q_heads, head_dim]")
    desc = cache_desc(k_cache)
    num_seqs, hq, d = q.shape
    max_blocks = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = max_blocks * desc.block_size
    if out is None:
        out = torch.empty((num_seqs, hq, d), dtype=out_dtype, device=q.device)
    _require(out.is_cuda and out.is_contiguous(), "out must be a contiguous CUDA tensor")
    need = paged_attention_workspace_bytes(num_seqs, hq, d, max_context_len, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().paged_attention_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), max_blocks, _ptr(context_lens), num_seqs, hq,
        int(max_context_len), float(scale), _ptr(out), _DTYPE_CODE.get(out.dtype, -1), ctypes.byref(desc),
        int(partition_size), _ptr(workspace), ws_bytes, _stream(stream)), "paged_attention_decode")
    return out


def paged_attention_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                               v_scales: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                               scale: float, out: torch.Tensor | None = None, max_context_len: int | None = None,
                               partition_size: int = 0, workspace: torch.Tensor | None = None,
                               out_dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """paged_attention_decode over float8_e4m3fn caches with one fp32 scale per (block, KV head)
    (paged_kv_append_rope_fp8); q is bf16 or fp16."""
    given = [q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens]
    given += [t for t in (out, workspace) if t is not None]
    dev = _one_device(given)
    if stream is not None or _current_device() != dev:
        with _context(dev, stream):
            return paged_attention_decode_fp8(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                                              scale, out, max_context_len, partition_size, workspace, out_dtype)
    shape, qshape, tables, cache_dt = k_cache.shape, q.shape, block_tables.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != cache_dt:
        raise ValueError("caches must be [num_blocks, num_kv_heads, block_size, head_dim], K as V")
    nb, hkv, bs, d = shape
    if len(qshape) != 3 or qshape[2] != d or (out is not None and out.shape != qshape):
        raise ValueError("q and out are [num_seqs, num_q_heads, head_dim]")
    num_seqs, hq, _ = qshape
    if block_tables.dtype != _I32 or len(tables) != 2 or tables[0] != num_seqs:
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks_per_seq]")
    if context_lens.dtype != _I32 or context_lens.shape != (num_seqs,):
        raise ValueError("context_lens must be int32 [num_seqs]")
    for s in (k_scales, v_scales):
        if s.dtype != _F32 or s.shape != (nb, hkv):
            raise ValueError("scales must be fp32 [num_blocks, num_kv_heads]")
    max_blocks = tables[1]
    max_context_len = max_blocks * bs if max_context_len is None else int(max_context_len)
    partition_size = int(partition_size)
    desc = CacheDesc(nb, hkv, bs, d, _DTYPE_CODE.get(cache_dt, -1))
    lib = _lib()

    if out is None:
        out = torch.empty(qshape, dtype=out_dtype, device=q.device)
    if workspace is None:
        need = lib.paged_attention_workspace_bytes(num_seqs, hq, d, max_context_len, partition_size)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                            workspace.numel() * workspace.element_size())
    st = lib.paged_attention_decode_fp8(
        q.data_ptr(), _DTYPE_CODE.get(q.dtype, -1), k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(),
        v_scales.data_ptr(), block_tables.data_ptr(), max_blocks, context_lens.data_ptr(), num_seqs, hq,
        max_context_len, float(scale), out.data_ptr(), _DTYPE_CODE.get(out.dtype, -1), desc, partition_size, ws_ptr,
        ws_bytes, _raw_stream(dev))
    if st != PKV_OK:
        raise PagedKVError(st, "paged_attention_decode_fp8")
    return out


def paged_attention_append_decode(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                  slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                                  out: torch.Tensor | None = None, max_context_len: int | None = None,
                                  partition_size: int = 0, workspace: torch.Tensor | None = None,
                                  out_dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """One decode step in one launch: write sequence s's new token (k_new[s], v_new[s]) to
    slot_mapping[s] -- the slot of its last context position -- then attend."""
    for t in (q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables, context_lens):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    _require(slot_mapping.dtype == torch.int64 and slot_mapping.numel() == q.shape[0],
             "slot_mapping: int64, one slot per sequence")
    desc = cache_desc(k_cache)
    num_seqs, hq, d = q.shape
    max_blocks = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = max_blocks * desc.block_size
    if out is None:
        out = torch.empty((num_seqs, hq, d), dtype=out_dtype, device=q.device)
    need = paged_attention_workspace_bytes(num_seqs, hq, d, max_context_len, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().paged_attention_append_decode(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        max_blocks, _ptr(context_lens), num_seqs, hq, int(max_context_len), float(scale), _ptr(out),
        _DTYPE_CODE.get(out.dtype, -1), ctypes.byref(desc), int(partition_size), _ptr(workspace), ws_bytes,
        _stream(stream)), "paged_attention_append_decode")
    return out


def paged_attention_grouped_workspace_bytes(num_seqs: int, num_q_heads: int, head_dim: int, max_context_len: int,
                                            max_prefix_len: int, partition_size: int = 0) -> int:
    return int(_lib().paged_attention_grouped_workspace_bytes(num_seqs, num_q_heads, head_dim, max_context_len,
                                                              max_prefix_len, partition_size))


def paged_attention_decode_grouped(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_tables: torch.Tensor, context_lens: torch.Tensor, group_starts: torch.Tensor,
                                   prefix_lens: torch.Tensor, scale: float, max_group_size: int,
                                   max_prefix_len: int, out: torch.Tensor | None = None,
                                   max_context_len: int | None = None, partition_size: int = 0,
                                   workspace: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                                   stream=None) -> torch.Tensor:
    """paged_attention_decode where the sequences group_starts[g] .. group_starts[g+1]-1
    share the blocks of their first prefix_lens[s] tokens with the group's first member;
    shared blocks are read once per (group, KV head)."""
    for t in (q, k_cache, v_cache, block_tables, context_lens, group_starts, prefix_lens):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    for t in (block_tables, context_lens, group_starts, prefix_lens):
        _require(t.dtype == torch.int32, "block_tables, context_lens, group_starts, prefix_lens must be int32")
    _require(q.dim() == 3 and block_tables.dim() == 2 and group_starts.dim() == 1, "bad shapes")
    desc = cache_desc(k_cache)
    num_seqs, hq, d = q.shape
    max_blocks = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = max_blocks * desc.block_size
    if out is None:
        out = torch.empty((num_seqs, hq, d), dtype=out_dtype, device=q.device)
    _require(out.is_cuda and out.is_contiguous(), "out must be a contiguous CUDA tensor")
    need = paged_attention_grouped_workspace_bytes(num_seqs, hq, d, max_context_len, max_prefix_len, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().paged_attention_decode_grouped(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), max_blocks, _ptr(context_lens), num_seqs, hq,
        int(max_context_len), _ptr(group_starts), group_starts.numel() - 1, int(max_group_size), _ptr(prefix_lens),
        int(max_prefix_len), float(scale), _ptr(out), _DTYPE_CODE.get(out.dtype, -1), ctypes.byref(desc),
        int(partition_size), _ptr(workspace), ws_bytes, _stream(stream)), "paged_attention_decode_grouped")
    return out


def paged_attention_append_decode_grouped(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                          slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                          block_tables: torch.Tensor, context_lens: torch.Tensor,
                                          group_starts: torch.Tensor, prefix_lens: torch.Tensor, scale: float,
                                          max_group_size: int, max_prefix_len: int, out: torch.Tensor | None = None,
                                          max_context_len: int | None = None, partition_size: int = 0,
                                          workspace: torch.Tensor | None = None,
                                          out_dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """One grouped decode step in one call: write sequence s's new token (k_new[s], v_new[s]) to
    slot_mapping[s] -- the slot of its last context position, past its shared prefix -- then
    paged_attention_decode_grouped."""
    for t in (q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables, context_lens, group_starts, prefix_lens):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    for t in (block_tables, context_lens, group_starts, prefix_lens):
        _require(t.dtype == torch.int32, "block_tables, context_lens, group_starts, prefix_lens must be int32")
    _require(slot_mapping.dtype == torch.int64 and slot_mapping.numel() == q.shape[0],
             "slot_mapping: int64, one slot per sequence")
    _require(q.dim() == 3 and block_tables.dim() == 2 and group_starts.dim() == 1, "bad shapes")
    desc = cache_desc(k_cache)
    num_seqs, hq, d = q.shape
    max_blocks = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = max_blocks * desc.block_size
    if out is None:
        out = torch.empty((num_seqs, hq, d), dtype=out_dtype, device=q.device)
    _require(out.is_cuda and out.is_contiguous(), "out must be a contiguous CUDA tensor")
    need = paged_attention_grouped_workspace_bytes(num_seqs, hq, d, max_context_len, max_prefix_len, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().paged_attention_append_decode_grouped(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        max_blocks, _ptr(context_lens), num_seqs, hq, int(max_context_len), _ptr(group_starts),
        group_starts.numel() - 1, int(max_group_size), _ptr(prefix_lens), int(max_prefix_len), float(scale),
        _ptr(out), _DTYPE_CODE.get(out.dtype, -1), ctypes.byref(desc), int(partition_size), _ptr(workspace),
        ws_bytes, _stream(stream)), "paged_attention_append_decode_grouped")
    return out


def paged_attention_decode_static(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                                  out: torch.Tensor, max_context_len: int, partition_size: int = 0,
                                  stream=None) -> torch.Tensor:
    """paged_attention_decode for callers that cannot allocate device memory: no
    workspace argument, the split-K partials go to the library's fixed 16 MiB
    device array (calls needing more raise PagedKVError(PKV_ERR_WORKSPACE))."""
    for t in (q, k_cache, v_cache, block_tables, context_lens, out):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    desc = cache_desc(k_cache)
    num_seqs, hq, _ = q.shape
    _check(_lib().paged_attention_decode_static(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
        num_seqs, hq, int(max_context_len), float(scale), _ptr(out), _DTYPE_CODE.get(out.dtype, -1),
        ctypes.byref(desc), int(partition_size), _stream(stream)), "paged_attention_decode_static")
    return out


def copy_blocks(k_caches: torch.Tensor | Sequence[torch.Tensor], v_caches: torch.Tensor | Sequence[torch.Tensor],
                src_dst_pairs: torch.Tensor, stream=None) -> None:
    """Copy-on-write block copy: for each (src, dst) pair, block dst := block src in every layer, K and V."""
    if isinstance(k_caches, torch.Tensor):
        k_caches = [k_caches]
    if isinstance(v_caches, torch.Tensor):
        v_caches = [v_caches]
    _require(len(k_caches) == len(v_caches) and len(k_caches) > 0, "need one K and one V cache per layer")
    for t in (*k_caches, *v_caches, src_dst_pairs):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    _require(src_dst_pairs.dtype == torch.int64 and (src_dst_pairs.numel() % 2 == 0),
             "src_dst_pairs must be int64 [n, 2]")
    desc = cache_desc(k_caches[0])
    n = len(k_caches)
    karr = (ctypes.c_void_p * n)(*[t.data_ptr() for t in k_caches])
    varr = (ctypes.c_void_p * n)(*[t.data_ptr() for t in v_caches])
    _check(_lib().copy_blocks(karr, varr, n, _ptr(src_dst_pairs), src_dst_pairs.numel() // 2, ctypes.byref(desc),
                              _stream(stream)), "copy_blocks")


def _ptr_array(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def copy_blocks_fp8(k_caches: torch.Tensor | Sequence[torch.Tensor], v_caches: torch.Tensor | Sequence[torch.Tensor],
                    k_scales: torch.Tensor | Sequence[torch.Tensor], v_scales: torch.Tensor | Sequence[torch.Tensor],
                    src_dst_pairs: torch.Tensor, stream=None) -> None:
    """copy_blocks for float8_e4m3fn caches: block dst := block src in every layer, K and V, with its scales."""
    k, v, ks, vs = ([t] if isinstance(t, torch.Tensor) else list(t) for t in (k_caches, v_caches, k_scales, v_scales))
    n = len(k)
    _require(n == len(v) == len(ks) == len(vs) > 0, "need one K and one V cache per layer, and their scales")
    caches, scales = k + v, ks + vs
    dev = _one_device(caches + scales + [src_dst_pairs])
    if stream is not None or _current_device() != dev:
        with _context(dev, stream):
            return copy_blocks_fp8(k, v, ks, vs, src_dst_pairs)
    desc = cache_desc(k[0])
    # whole tensors of one size and type: nothing lies outside them
    _require(len(set(map(_numel, caches))) == 1 == len(set(map(_dtype_of, caches))), "the caches differ")
    _require(set(map(_numel, scales)) == {desc.num_blocks * desc.num_kv_heads} and
             set(map(_dtype_of, scales)) == {_F32}, "scales must be fp32 [num_blocks, num_kv_heads]")
    _require(src_dst_pairs.dtype == _I64 and src_dst_pairs.numel() % 2 == 0, "src_dst_pairs must be int64 [n, 2]")
    ptrs = array.array("Q", map(torch.Tensor.data_ptr, caches + scales))  # the four host arrays, one after the other
    at, step = ptrs.buffer_info()[0], n * ptrs.itemsize
    _check(_lib().copy_blocks_fp8(at, at + step, at + 2 * step, at + 3 * step, n, src_dst_pairs.data_ptr(),
                                  src_dst_pairs.numel() // 2, desc, _raw_stream(dev)), "copy_blocks_fp8")


def swap_blocks(src_k: torch.Tensor | Sequence[torch.Tensor], src_v: torch.Tensor | Sequence[torch.Tensor],
                dst_k: torch.Tensor | Sequence[torch.Tensor], dst_v: torch.Tensor | Sequence[torch.Tensor],
                src_dst_pairs: torch.Tensor, stream=None) -> None:
    """Move whole blocks src -> dst between two pools (GPU or pinned host memory), every layer, K and V."""
    src_k, src_v, dst_k, dst_v = ([t] if isinstance(t, torch.Tensor) else list(t) for t in (src_k, src_v, dst_k, dst_v))
    _require(len(src_k) == len(src_v) == len(dst_k) == len(dst_v) > 0, "one K and one V pool per layer on each side")
    for t in (*src_k, *src_v, *dst_k, *dst_v):
        _require(t.is_contiguous() and (t.is_cuda or t.is_pinned()), "pools must be contiguous, on the GPU or pinned")
    _require(src_dst_pairs.dtype == torch.int64 and src_dst_pairs.numel() % 2 == 0, "src_dst_pairs: int64 [n, 2]")
    _require(src_dst_pairs.is_cuda or src_dst_pairs.is_pinned(), "src_dst_pairs must be GPU-addressable")
    desc = cache_desc(src_k[0])
    _check(_lib().swap_blocks(_ptr_array(src_k), _ptr_array(src_v), src_k[0].shape[0], _ptr_array(dst_k),
                              _ptr_array(dst_v), dst_k[0].shape[0], len(src_k), _ptr(src_dst_pairs),
                              src_dst_pairs.numel() // 2, ctypes.byref(desc), _stream(stream)), "swap_blocks")


def compact_tokens(src_slots: torch.Tensor, dst_slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   stream=None) -> None:
    """Move the K/V rows of every head from slot src_slots[i] to slot dst_slots[i]."""
    for t in (src_slots, dst_slots, k_cache, v_cache):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    _require(src_slots.dtype == torch.int64 and dst_slots.dtype == torch.int64 and
             src_slots.numel() == dst_slots.numel(), "src_slots/dst_slots: int64 of equal length")
    desc = cache_desc(k_cache)
    _check(_lib().compact_tokens(_ptr(src_slots), _ptr(dst_slots), src_slots.numel(), _ptr(k_cache), _ptr(v_cache),
                                 ctypes.byref(desc), _stream(stream)), "compact_tokens")


def wait_selftest(limit_us: int = 50_000, stream=None) -> None:
    """pkv_wait_selftest: one CTA's bounded wait on a phase nothing completes
    runs out after limit_us and records PKV_DEVERR_TIMEOUT (read it with
    check_device_error)."""
    _check(_lib().pkv_wait_selftest(int(limit_us), _stream(stream)), "pkv_wait_selftest")


def check_device_error(stream=None) -> int:
    """Synchronise the stream; return and clear the first device-side error code (0: none)."""
    code = ctypes.c_int32(0)
    st = _lib().pkv_check_device_error(_stream(stream), ctypes.byref(code))
    if st not in (PKV_OK, PKV_ERR_DEVICE_METADATA):
        raise PagedKVError(st, "pkv_check_device_error")
    return int(code.value)
