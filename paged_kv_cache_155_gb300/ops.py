"""Thin PyTorch binding of libpagedkv: same names as the C ABI, argument
marshalling only.  Tensors supply device pointers and shapes; the current
CUDA stream of the tensors' device is passed as the stream.  Every step runs
in the library's kernels; if the library is missing the calls raise.

``prepare_*`` variants check and marshal a call's arguments once and return a
``PreparedCall``; calling it enqueues the same library call again on the
current stream (a serving loop that reuses its buffers pays the argument
checks once, not per step).

Cache tensors: ``k_cache`` / ``v_cache`` are [num_blocks, num_kv_heads,
block_size, head_dim] views sharing one block stride, normally the two
halves ``kv[:, 0]`` / ``kv[:, 1]`` of a pool ``kv`` of shape
[num_blocks, 2, num_kv_heads, block_size, head_dim] ("KV Cache与PagedAttention深度解析"
§4.3 and §5.1).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from ._lib import DEVERR, PagedKVError, lib

F16, BF16, INT8 = 0, 1, 2
_workspaces = {}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}: fp16 or bf16 expected")


_raw_stream_getter = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# the current device's index (without torch's initialisation check: a prepared call's
# tensors are on a device already)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _raw_stream(device_index: int) -> int:
    """cudaStream_t of the device's current stream, as an integer."""
    if _raw_stream_getter is not None:
        return _raw_stream_getter(device_index)
    return torch.cuda.current_stream(device_index).cuda_stream


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(_raw_stream(t.device.index if t.device.index is not None
                                       else torch.cuda.current_device()))


class PreparedCall:
    """One library call whose arguments were checked and marshalled once.

    Calling it enqueues the same call on the current stream of its device and
    returns the call's output tensor (or None).  It holds the tensors it was
    prepared with; they must keep their storage, while their contents may change
    between calls (new queries and rows, new context lengths within the bound
    given at preparation).  Its output and workspace are its own: calls of one
    PreparedCall must not overlap on the GPU, and it must stay alive until they are done."""
    __slots__ = ("_fn", "_args", "_dev", "_what", "_tensors", "_result", "_calls")

    @property
    def result(self):
        """What the call returns (its output tensors, written by each call)."""
        return self._result

    def __init__(self, what: str, args: tuple, device: torch.device, tensors: tuple, result=None):
        self._fn = getattr(lib(), what)
        self._args = args
        self._dev = device.index if device.index is not None else torch.cuda.current_device()
        self._what = what
        self._tensors = tensors
        self._result = result
        self._calls = 0

    def _typed_args(self) -> tuple:
        """The arguments as the ctypes values that the call converts them to."""
        return tuple(ty(a) if issubclass(ty, ctypes._SimpleCData) and type(a) in (int, float, bool, type(None)) else a
                     for ty, a in zip(self._fn.argtypes, self._args))

    def __call__(self):
        if self._calls < 2:
            # from the second call on the arguments are kept converted (26 of them: 2.5 us a call
            # instead of 3.5); a single call would pay more for it than it saves
            self._calls += 1
            if self._calls == 2:
                self._args = self._typed_args()
        if _current_device() != self._dev:  # the library launches on the current device
            with torch.cuda.device(self._dev):
                st = self._fn(*self._args, _raw_stream(self._dev))
        else:
            st = self._fn(*self._args, _raw_stream(self._dev))
        if st != 0:
            raise PagedKVError(self._what, st)
        return self._result


def _check(status: int, what: str):
    if status != 0:
        raise PagedKVError(what, status)


def _cache_dtype_code(t: torch.Tensor) -> int:
    return INT8 if t.dtype == torch.int8 else _dtype_code(t)


def _cache_geometry(k_cache: torch.Tensor, v_cache: torch.Tensor):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache/v_cache must be [num_blocks, num_kv_heads, block_size, head_dim]")
    if k_cache.stride() != v_cache.stride() or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must share dtype and strides")
    nb, hkv, bs, d = k_cache.shape
    if k_cache.stride()[1:] != (bs * d, d, 1):
        raise ValueError("each block of k_cache/v_cache must be a dense [num_kv_heads, block_size, head_dim]")
    return nb, hkv, bs, d, k_cache.stride(0)


def split_pool(kv: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """K and V halves of a pool [num_blocks, 2, num_kv_heads, block_size, head_dim]."""
    if kv.dim() != 5 or kv.shape[1] != 2 or not kv.is_contiguous():
        raise ValueError("pool must be a contiguous [num_blocks, 2, num_kv_heads, block_size, head_dim]")
    return kv[:, 0], kv[:, 1]


def reshape_and_cache(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                      k_cache: torch.Tensor, v_cache: torch.Tensor) -> None:
    """Write new K/V rows [T, Hkv, d] into their slots (bit-exact); slot < 0 skips."""
    prepare_reshape_and_cache(k_new, v_new, slot_mapping, k_cache, v_cache)()


def prepare_reshape_and_cache(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                              k_cache: torch.Tensor, v_cache: torch.Tensor) -> PreparedCall:
    """reshape_and_cache, checked and marshalled once (see PreparedCall)."""
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    t = int(k_new.shape[0])
    if k_new.shape != (t, hkv, d) or v_new.shape != k_new.shape:
        raise ValueError(f"k_new/v_new must be [T, {hkv}, {d}]")
    if not (k_new.is_contiguous() and v_new.is_contiguous() and slot_mapping.is_contiguous()):
        raise ValueError("k_new, v_new and slot_mapping must be contiguous")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != t:
        raise ValueError("slot_mapping must be int64 [T]")
    if k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype:
        raise ValueError("k_new/v_new dtype must match the cache")
    args = (k_new.data_ptr(), v_new.data_ptr(), slot_mapping.data_ptr(), t, k_cache.data_ptr(),
            v_cache.data_ptr(), nb, stride, hkv, d, bs, _dtype_code(k_cache))
    return PreparedCall("pkv_reshape_and_cache", args, k_cache.device,
                        (k_new, v_new, slot_mapping, k_cache, v_cache))


def decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                           max_context_len, partition_size=0) -> int:
    n = lib().pkv_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                         block_size, max_context_len, partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError("pkv_decode_workspace_bytes", 1)
    return int(n)


def _workspace(device: torch.device, nbytes: int) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    key = (device.type, device.index)
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _workspaces[key] = buf
    return buf


def paged_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor,
                           scale: Optional[float] = None, out: Optional[torch.Tensor] = None, *,
                           max_context_len: Optional[int] = None, partition_size: int = 0,
                           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[i, hq] = softmax(scale * q[i, hq] . K_i^T) V_i over the paged cache.

    q, out: [num_seqs, num_q_heads, head_dim]; block_tables int32 [num_seqs, max_blocks];
    context_lens int32 [num_seqs].  ``max_context_len`` (a host int) bounds
    context_lens; if omitted it is read back from the device (a synchronisation).
    """
    return prepare_paged_attention_decode(q, k_cache, v_cache, block_tables, context_lens, scale,
                                          out, max_context_len=max_context_len,
                                          partition_size=partition_size, workspace=workspace)()


def prepare_paged_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_tables: torch.Tensor, context_lens: torch.Tensor,
                                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                                   *, max_context_len: Optional[int] = None, partition_size: int = 0,
                                   workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """paged_attention_decode, checked and marshalled once (see PreparedCall); the
    call returns ``out``.  Later context lengths must stay within max_context_len."""
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    if q.dim() != 3 or q.shape[2] != d or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous [num_seqs, num_q_heads, {d}]")
    b, hq = int(q.shape[0]), int(q.shape[1])
    if q.dtype != k_cache.dtype:
        raise ValueError("q dtype must match the cache")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b \
            or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks_per_seq]")
    if context_lens.dtype != torch.int32 or context_lens.numel() != b or not context_lens.is_contiguous():
        raise ValueError("context_lens must be a contiguous int32 [num_seqs]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_context_len is None:
        max_context_len = int(context_lens.max().item()) if b else 0
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must match q")
    need = decode_workspace_bytes(b, hq, hkv, d, bs, max_context_len, partition_size)
    if workspace is None:
        workspace = _workspace(q.device, need)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), nb, stride, block_tables.data_ptr(),
            int(block_tables.shape[1]), context_lens.data_ptr(), int(max_context_len), b, hq, hkv, d,
            bs, float(scale), out.data_ptr(), ws_ptr, ws_bytes, int(partition_size), _dtype_code(q))
    return PreparedCall("pkv_paged_attention_decode", args, q.device,
                        (q, k_cache, v_cache, block_tables, context_lens, out, workspace), out)


def shared_prefix_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                  prefix_len, max_context_len, partition_size=0) -> int:
    n = lib().pkv_shared_prefix_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                block_size, prefix_len, max_context_len,
                                                partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError("pkv_shared_prefix_workspace_bytes", 1)
    return int(n)


def paged_attention_decode_shared_prefix(q: torch.Tensor, k_cache: torch.Tensor,
                                         v_cache: torch.Tensor, prefix_block_table: torch.Tensor,
                                         prefix_len: int, block_tables: torch.Tensor,
                                         context_lens: torch.Tensor, scale: Optional[float] = None,
                                         out: Optional[torch.Tensor] = None, *,
                                         max_context_len: Optional[int] = None,
                                         partition_size: int = 0,
                                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attention_decode for a batch that shares its first prefix_len tokens
    (prefix_block_table holds their blocks): the prefix is attended by all query
    rows together as dense tiles, beside each sequence's suffix, then a merge."""
    return prepare_paged_attention_decode_shared_prefix(
        q, k_cache, v_cache, prefix_block_table, prefix_len, block_tables, context_lens, scale, out,
        max_context_len=max_context_len, partition_size=partition_size, workspace=workspace)()


def prepare_paged_attention_decode_shared_prefix(
        q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
        prefix_block_table: torch.Tensor, prefix_len: int, block_tables: torch.Tensor,
        context_lens: torch.Tensor, scale: Optional[float] = None,
        out: Optional[torch.Tensor] = None, *, max_context_len: Optional[int] = None,
        partition_size: int = 0, workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """paged_attention_decode_shared_prefix, checked and marshalled once (see
    PreparedCall); the call returns ``out``."""
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    if q.dim() != 3 or q.shape[2] != d or not q.is_contiguous() or q.dtype != k_cache.dtype:
        raise ValueError(f"q must be a contiguous [num_seqs, num_q_heads, {d}] of the cache dtype")
    b, hq = int(q.shape[0]), int(q.shape[1])
    if prefix_block_table.dtype != torch.int32 or not prefix_block_table.is_contiguous():
        raise ValueError("prefix_block_table must be a contiguous int32 tensor")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks_per_seq]")
    if context_lens.dtype != torch.int32 or context_lens.numel() != b:
        raise ValueError("context_lens must be int32 [num_seqs]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_context_len is None:
        max_context_len = int(context_lens.max().item())
    if out is None:
        out = torch.empty_like(q)
    need = shared_prefix_workspace_bytes(b, hq, hkv, d, bs, prefix_len, max_context_len,
                                         partition_size)
    if workspace is None:
        workspace = _workspace(q.device, need)
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), nb, stride,
            prefix_block_table.data_ptr(), int(prefix_len), block_tables.data_ptr(),
            int(block_tables.shape[1]), context_lens.data_ptr(), int(max_context_len), b, hq, hkv, d,
            bs, float(scale), out.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), int(partition_size), _dtype_code(q))
    return PreparedCall("pkv_paged_attention_decode_shared_prefix", args, q.device,
                        (q, k_cache, v_cache, prefix_block_table, block_tables, context_lens, out,
                         workspace), out)


def prefill_workspace_bytes(num_rows, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                            max_query_len, max_context_len, kv_splits=0) -> int:
    n = lib().pkv_prefill_workspace_bytes(num_rows, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                          block_size, max_query_len, max_context_len, kv_splits)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError("pkv_prefill_workspace_bytes", 1)
    return int(n)


def paged_attention_prefill(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, query_start: torch.Tensor,
                            context_lens: torch.Tensor, scale: Optional[float] = None,
                            out: Optional[torch.Tensor] = None, *, max_query_len: int,
                            max_context_len: int, kv_splits: int = 0,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Chunked prefill attention: q [num_rows, Hq, d] holds every sequence's chunk
    (sequence i owns rows query_start[i]:query_start[i+1], whose K/V are already in
    the cache as its last tokens); row j of chunk i attends causally to tokens
    0 .. context_lens[i] - chunk_i + j.  max_query_len / max_context_len are host bounds."""
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    if q.dim() != 3 or q.shape[2] != d or not q.is_contiguous() or q.dtype != k_cache.dtype:
        raise ValueError(f"q must be a contiguous [num_rows, num_q_heads, {d}] of the cache dtype")
    rows, hq = int(q.shape[0]), int(q.shape[1])
    b = int(context_lens.numel())
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b \
            or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks_per_seq]")
    if query_start.dtype != torch.int32 or query_start.numel() != b + 1 \
            or not query_start.is_contiguous():
        raise ValueError("query_start must be a contiguous int32 [num_seqs + 1]")
    if context_lens.dtype != torch.int32 or not context_lens.is_contiguous():
        raise ValueError("context_lens must be a contiguous int32 [num_seqs]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must match q")
    need = prefill_workspace_bytes(rows, b, hq, hkv, d, bs, max_query_len, max_context_len,
                                   kv_splits)
    if workspace is None:
        workspace = _workspace(q.device, need)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().pkv_paged_attention_prefill(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), nb, stride, block_tables.data_ptr(),
        int(block_tables.shape[1]), query_start.data_ptr(), context_lens.data_ptr(), rows,
        int(max_query_len), int(max_context_len), b, hq, hkv, d, bs, float(scale), out.data_ptr(),
        ws_ptr, ws_bytes, int(kv_splits), _dtype_code(q), _stream(q))
    _check(st, "pkv_paged_attention_prefill")
    return out


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, src_dst_pairs: torch.Tensor) -> None:
    """Copy K and V of block src over block dst for each row (src, dst) of an int64 [n, 2]."""
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2 \
            or not src_dst_pairs.is_contiguous():
        raise ValueError("src_dst_pairs must be a contiguous int64 [n, 2]")
    if src_dst_pairs.device.type == "cpu":
        raise ValueError("src_dst_pairs must be on the device")
    st = lib().pkv_copy_blocks(k_cache.data_ptr(), v_cache.data_ptr(), nb, stride, hkv, d, bs,
                               src_dst_pairs.data_ptr(), int(src_dst_pairs.shape[0]),
                               _cache_dtype_code(k_cache), _stream(k_cache))
    _check(st, "pkv_copy_blocks")


# ---------------------------------------------------------------------------
# INT8 cache with per-channel scales ("KV Cache从原理到实战" §5.2)
# ---------------------------------------------------------------------------

def _check_int8_cache(k_cache, v_cache, k_scale, v_scale):
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    if k_cache.dtype != torch.int8:
        raise ValueError("k_cache/v_cache must be int8")
    for name, sc in (("k_scale", k_scale), ("v_scale", v_scale)):
        if sc.dtype != torch.float32 or sc.shape != (hkv, d) or not sc.is_contiguous() \
                or sc.device != k_cache.device:
            raise ValueError(f"{name} must be a contiguous float32 [{hkv}, {d}] on the cache's device")
    return nb, hkv, bs, d, stride


def reshape_and_cache_int8(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                           k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                           v_scale: torch.Tensor) -> None:
    """Quantise new K/V rows [T, Hkv, d] (fp16/bf16) with per-channel scales [Hkv, d]
    and write the codes into their slots of an INT8 cache; slot < 0 skips."""
    prepare_reshape_and_cache_int8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale)()


def prepare_reshape_and_cache_int8(k_new: torch.Tensor, v_new: torch.Tensor,
                                   slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, k_scale: torch.Tensor,
                                   v_scale: torch.Tensor) -> PreparedCall:
    """reshape_and_cache_int8, checked and marshalled once (see PreparedCall)."""
    nb, hkv, bs, d, stride = _check_int8_cache(k_cache, v_cache, k_scale, v_scale)
    t = int(k_new.shape[0])
    if k_new.shape != (t, hkv, d) or v_new.shape != k_new.shape or v_new.dtype != k_new.dtype:
        raise ValueError(f"k_new/v_new must be [T, {hkv}, {d}] of one dtype")
    if not (k_new.is_contiguous() and v_new.is_contiguous() and slot_mapping.is_contiguous()):
        raise ValueError("k_new, v_new and slot_mapping must be contiguous")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != t:
        raise ValueError("slot_mapping must be int64 [T]")
    args = (k_new.data_ptr(), v_new.data_ptr(), slot_mapping.data_ptr(), t, k_cache.data_ptr(),
            v_cache.data_ptr(), nb, stride, hkv, d, bs, k_scale.data_ptr(), v_scale.data_ptr(),
            _dtype_code(k_new))
    return PreparedCall("pkv_reshape_and_cache_int8", args, k_cache.device,
                        (k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale))


def decode_int8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                max_context_len, partition_size=0) -> int:
    n = lib().pkv_decode_int8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                              block_size, max_context_len, partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError("pkv_decode_int8_workspace_bytes", 1)
    return int(n)


def paged_attention_decode_int8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                k_scale: torch.Tensor, v_scale: torch.Tensor,
                                block_tables: torch.Tensor, context_lens: torch.Tensor,
                                scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                                *, max_context_len: Optional[int] = None, partition_size: int = 0,
                                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attention_decode over an INT8 cache whose values are code * scale[h][channel];
    q and out fp16 or bf16."""
    return prepare_paged_attention_decode_int8(
        q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, out,
        max_context_len=max_context_len, partition_size=partition_size, workspace=workspace)()


def prepare_paged_attention_decode_int8(q: torch.Tensor, k_cache: torch.Tensor,
                                        v_cache: torch.Tensor, k_scale: torch.Tensor,
                                        v_scale: torch.Tensor, block_tables: torch.Tensor,
                                        context_lens: torch.Tensor, scale: Optional[float] = None,
                                        out: Optional[torch.Tensor] = None, *,
                                        max_context_len: Optional[int] = None,
                                        partition_size: int = 0,
                                        workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """paged_attention_decode_int8, checked and marshalled once (see PreparedCall); the
    call returns ``out``."""
    nb, hkv, bs, d, stride = _check_int8_cache(k_cache, v_cache, k_scale, v_scale)
    if q.dim() != 3 or q.shape[2] != d or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous [num_seqs, num_q_heads, {d}]")
    b, hq = int(q.shape[0]), int(q.shape[1])
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b \
            or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks_per_seq]")
    if context_lens.dtype != torch.int32 or context_lens.numel() != b or not context_lens.is_contiguous():
        raise ValueError("context_lens must be a contiguous int32 [num_seqs]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_context_len is None:
        max_context_len = int(context_lens.max().item()) if b else 0
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must match q")
    need = decode_int8_workspace_bytes(b, hq, hkv, d, bs, max_context_len, partition_size)
    if workspace is None:
        workspace = _workspace(q.device, need)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), nb, stride, block_tables.data_ptr(), int(block_tables.shape[1]),
            context_lens.data_ptr(), int(max_context_len), b, hq, hkv, d, bs, float(scale),
            out.data_ptr(), ws_ptr, ws_bytes, int(partition_size), _dtype_code(q))
    return PreparedCall("pkv_paged_attention_decode_int8", args, q.device,
                        (q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, out,
                         workspace), out)


# ---------------------------------------------------------------------------
# Rotary positions with the cache write
# ---------------------------------------------------------------------------

def _one_device(anchor: torch.Tensor, **tensors) -> None:
    """Every given tensor is on the anchor's device, a CUDA device."""
    for name, t in tensors.items():
        if t is not None and t.device != anchor.device:
            raise ValueError(f"{name} must be on {anchor.device}, not {t.device}")
    if anchor.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")


def _int32(**values) -> None:
    """The C ABI's int arguments: ctypes would cut a larger value to its low 32 bits."""
    for name, v in values.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name} must fit 32 bits")


def _token_rows(t: torch.Tensor, name: str, tokens: int, heads: Optional[int], d: int) -> Tuple[int, int]:
    """(heads, elements between tokens) of a [tokens, heads, d] tensor dense within a token."""
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [{tokens}, {'num_q_heads' if heads is None else heads}, {d}]")
    h = int(t.shape[1])
    if t.stride(2) != 1 or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name} must be dense within a token")
    stride = int(t.stride(0)) if tokens > 1 else h * d
    if stride < h * d or stride % 8:
        raise ValueError(f"{name}'s tokens must be a multiple of 8 elements apart and not overlap")
    return h, stride


def _rope_args(q, k_new, v_new, positions, inv_freq, slot_mapping, k_cache, v_cache, q_out, axis_of_pair,
               interleaved, geometry):
    nb, hkv, bs, d, stride = geometry
    if q.dim() != 3:
        raise ValueError(f"q must be [T, num_q_heads, {d}]")
    t = int(q.shape[0])
    hq, q_stride = _token_rows(q, "q", t, None, d)
    _, k_stride = _token_rows(k_new, "k_new", t, hkv, d)
    _, v_stride = _token_rows(v_new, "v_new", t, hkv, d)
    if k_new.dtype != q.dtype or v_new.dtype != q.dtype:
        raise ValueError("q, k_new and v_new must have one dtype")
    if q_out is None:
        q_out = torch.empty((t, hq, d), dtype=q.dtype, device=q.device)
    if q_out.dtype != q.dtype:
        raise ValueError("q_out must have q's dtype")
    _, q_out_stride = _token_rows(q_out, "q_out", t, hq, d)
    if positions.dtype != torch.int64 or positions.dim() not in (1, 2) or positions.shape[-1] != t \
            or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int64 [T] or [num_axes, T]")
    axes = int(positions.shape[0]) if positions.dim() == 2 else 1
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 [rotary_dim / 2]")
    if axis_of_pair is not None and (axis_of_pair.dtype != torch.int32 or axis_of_pair.shape != inv_freq.shape
                                     or not axis_of_pair.is_contiguous()):
        raise ValueError("axis_of_pair must be a contiguous int32 [rotary_dim / 2]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != t or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 [T]")
    _one_device(k_cache, q=q, k_new=k_new, v_new=v_new, positions=positions, inv_freq=inv_freq,
                slot_mapping=slot_mapping, v_cache=v_cache, q_out=q_out, axis_of_pair=axis_of_pair)
    args = (q.data_ptr(), q_stride, k_new.data_ptr(), k_stride, v_new.data_ptr(), v_stride, positions.data_ptr(),
            axes, None if axis_of_pair is None else axis_of_pair.data_ptr(), inv_freq.data_ptr(),
            2 * int(inv_freq.numel()), int(bool(interleaved)), slot_mapping.data_ptr(), t, q_out.data_ptr(),
            q_out_stride, k_cache.data_ptr(), v_cache.data_ptr(), nb, stride, hq, hkv, d, bs)
    return args, (q, k_new, v_new, positions, inv_freq, slot_mapping, k_cache, v_cache, q_out, axis_of_pair), q_out


def rope_reshape_and_cache(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                           inv_freq: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, q_out: Optional[torch.Tensor] = None, *,
                           axis_of_pair: Optional[torch.Tensor] = None, interleaved: bool = False) -> torch.Tensor:
    """Rotate q [T, Hq, d] and k_new [T, Hkv, d] by their positions and write the rotated
    K rows and the V rows into their slots; returns the rotated q (``q_out``).

    positions: int64 [T], or [num_axes, T] (up to four) with axis_of_pair int32
    [rotary_dim/2] naming the axis that each pair of channels follows; inv_freq:
    float64 [rotary_dim/2], radians per position.  Pairs are channels (i, i +
    rotary_dim/2), or (2i, 2i + 1) when ``interleaved``; channels from rotary_dim on
    are copied.  q, k_new and v_new may be views of one projection's rows (dense
    within a token).  slot < 0 writes no cache row.  q_out may be q."""
    return prepare_rope_reshape_and_cache(q, k_new, v_new, positions, inv_freq, slot_mapping, k_cache, v_cache, q_out,
                                          axis_of_pair=axis_of_pair, interleaved=interleaved)()


def prepare_rope_reshape_and_cache(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                   positions: torch.Tensor, inv_freq: torch.Tensor, slot_mapping: torch.Tensor,
                                   k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   q_out: Optional[torch.Tensor] = None, *,
                                   axis_of_pair: Optional[torch.Tensor] = None,
                                   interleaved: bool = False) -> PreparedCall:
    """rope_reshape_and_cache, checked and marshalled once (see PreparedCall)."""
    geometry = _cache_geometry(k_cache, v_cache)
    if q.dtype != k_cache.dtype:
        raise ValueError("q, k_new and v_new must have the cache's dtype")
    args, held, q_out = _rope_args(q, k_new, v_new, positions, inv_freq, slot_mapping, k_cache, v_cache, q_out,
                                   axis_of_pair, interleaved, geometry)
    return PreparedCall("pkv_rope_reshape_and_cache", args + (_dtype_code(q),), k_cache.device, held, q_out)


def rope_reshape_and_cache_int8(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                                inv_freq: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                                v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                                q_out: Optional[torch.Tensor] = None, *,
                                axis_of_pair: Optional[torch.Tensor] = None,
                                interleaved: bool = False) -> torch.Tensor:
    """rope_reshape_and_cache into an INT8 cache: the rotated K rows and the V rows are
    quantised with the per-channel scales [Hkv, d]."""
    return prepare_rope_reshape_and_cache_int8(q, k_new, v_new, positions, inv_freq, slot_mapping, k_cache, v_cache,
                                               k_scale, v_scale, q_out, axis_of_pair=axis_of_pair,
                                               interleaved=interleaved)()


def prepare_rope_reshape_and_cache_int8(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                        positions: torch.Tensor, inv_freq: torch.Tensor, slot_mapping: torch.Tensor,
                                        k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                                        v_scale: torch.Tensor, q_out: Optional[torch.Tensor] = None, *,
                                        axis_of_pair: Optional[torch.Tensor] = None,
                                        interleaved: bool = False) -> PreparedCall:
    """rope_reshape_and_cache_int8, checked and marshalled once (see PreparedCall)."""
    geometry = _check_int8_cache(k_cache, v_cache, k_scale, v_scale)
    args, held, q_out = _rope_args(q, k_new, v_new, positions, inv_freq, slot_mapping, k_cache, v_cache, q_out,
                                   axis_of_pair, interleaved, geometry)
    return PreparedCall("pkv_rope_reshape_and_cache_int8",
                        args + (k_scale.data_ptr(), v_scale.data_ptr(), _dtype_code(q)), k_cache.device,
                        held + (k_scale, v_scale), q_out)


# ---------------------------------------------------------------------------
# Scored attention: capped and biased scores, windows and starts, weights
# ---------------------------------------------------------------------------

def decode_scored_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len,
                                  window=0, want_weights=False, int8=False, partition_size=0) -> int:
    n = lib().pkv_decode_scored_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                max_context_len, window, int(want_weights), int(int8),
                                                partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError("pkv_decode_scored_workspace_bytes", 1)
    return int(n)


def _own_workspace(device: torch.device, nbytes: int, given: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """The caller's workspace, or one of this call's own: two prepared calls, or two
    captured graphs, never meet in it."""
    if given is not None:
        if given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be contiguous and on the tensors' device")
        return given
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _check_scores(softcap, slopes, window, hq):
    if softcap != 0.0 and not 1e-3 <= softcap <= 1e6:
        raise ValueError("softcap must be 0 or in [1e-3, 1e6]")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.numel() != hq or not slopes.is_contiguous()):
        raise ValueError("slopes must be a contiguous float32 [num_q_heads]")
    if window < 0:
        raise ValueError("window must not be negative")


def _prepare_decode_scored(what, q, k_cache, v_cache, scales, block_tables, context_lens, scale, out, softcap, slopes,
                           window, starts, weights, weights_out, max_context_len, partition_size, workspace):
    nb, hkv, bs, d, stride = _check_int8_cache(k_cache, v_cache, *scales) if scales else _cache_geometry(k_cache, v_cache)
    if q.dim() != 3 or q.shape[2] != d or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous [num_seqs, num_q_heads, {d}]")
    b, hq = int(q.shape[0]), int(q.shape[1])
    if not scales and q.dtype != k_cache.dtype:
        raise ValueError("q dtype must match the cache")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b \
            or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks_per_seq]")
    if context_lens.dtype != torch.int32 or context_lens.numel() != b or not context_lens.is_contiguous():
        raise ValueError("context_lens must be a contiguous int32 [num_seqs]")
    _check_scores(softcap, slopes, window, hq)
    _int32(window=window, partition_size=partition_size, max_context_len=max_context_len or 0)
    if starts is not None and (starts.dtype != torch.int32 or starts.numel() != b or not starts.is_contiguous()):
        raise ValueError("starts must be a contiguous int32 [num_seqs]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_context_len is None:
        max_context_len = int(context_lens.max().item()) if b else 0
    if weights is not None and weights_out is None:
        raise ValueError("weights need weights_out (which may be the same tensor)")
    for name, t in (("weights", weights), ("weights_out", weights_out)):
        if t is not None and (t.dtype != torch.float32 or t.dim() != 3 or tuple(t.shape[:2]) != (b, hkv)
                              or t.shape[2] < max_context_len or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 [num_seqs, num_kv_heads, >= max_context_len]")
    if weights is not None and weights.shape != weights_out.shape:
        raise ValueError("weights and weights_out must have one shape")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must match q")
    _one_device(q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables, context_lens=context_lens, out=out,
                slopes=slopes, starts=starts, weights=weights, weights_out=weights_out)
    with torch.cuda.device(q.device):
        need = decode_scored_workspace_bytes(b, hq, hkv, d, bs, max_context_len, window, weights_out is not None,
                                             bool(scales), partition_size)
    workspace = _own_workspace(q.device, need, workspace)
    ptr = lambda t: None if t is None else t.data_ptr()
    args = [q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()]
    args += [t.data_ptr() for t in scales]
    args += [nb, stride, block_tables.data_ptr(), int(block_tables.shape[1]), context_lens.data_ptr(),
             int(max_context_len), b, hq, hkv, d, bs, float(scale), float(softcap), ptr(slopes), int(window), ptr(starts)]
    if not scales:
        args += [ptr(weights), ptr(weights_out), 0 if weights_out is None else int(weights_out.shape[2])]
    args += [out.data_ptr(), ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
             int(partition_size), _dtype_code(q)]
    return PreparedCall(what, tuple(args), q.device,
                        (q, k_cache, v_cache, scales, block_tables, context_lens, out, slopes, starts, weights,
                         weights_out, workspace), out)


def paged_attention_decode_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, *,
                                  softcap: float = 0.0, slopes: Optional[torch.Tensor] = None, window: int = 0,
                                  starts: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                                  weights_out: Optional[torch.Tensor] = None, max_context_len: Optional[int] = None,
                                  partition_size: int = 0, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attention_decode with capped scores (softcap * tanh(x / softcap)), a distance
    bias (slopes fp32 [Hq] times t - position), the last ``window`` tokens only, and a
    first visible token per sequence (starts int32 [B]); a sequence that sees nothing
    gets zeros.  ``weights_out`` fp32 [B, Hkv, W] receives ``weights`` (None: zeros) plus
    each context token's softmax weight summed over its KV head's query heads; it may be
    ``weights`` itself."""
    return prepare_paged_attention_decode_scored(
        q, k_cache, v_cache, block_tables, context_lens, scale, out, softcap=softcap, slopes=slopes, window=window,
        starts=starts, weights=weights, weights_out=weights_out, max_context_len=max_context_len,
        partition_size=partition_size, workspace=workspace)()


def prepare_paged_attention_decode_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                          block_tables: torch.Tensor, context_lens: torch.Tensor,
                                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None, *,
                                          softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                                          window: int = 0, starts: Optional[torch.Tensor] = None,
                                          weights: Optional[torch.Tensor] = None,
                                          weights_out: Optional[torch.Tensor] = None,
                                          max_context_len: Optional[int] = None, partition_size: int = 0,
                                          workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """paged_attention_decode_scored, checked and marshalled once (see PreparedCall); the
    call returns ``out``.  Without ``workspace`` it holds one of its own."""
    return _prepare_decode_scored("pkv_paged_attention_decode_scored", q, k_cache, v_cache, (), block_tables,
                                  context_lens, scale, out, softcap, slopes, window, starts, weights, weights_out,
                                  max_context_len, partition_size, workspace)


def paged_attention_decode_scored_int8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                       k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                                       context_lens: torch.Tensor, scale: Optional[float] = None,
                                       out: Optional[torch.Tensor] = None, *, softcap: float = 0.0,
                                       slopes: Optional[torch.Tensor] = None, window: int = 0,
                                       starts: Optional[torch.Tensor] = None, max_context_len: Optional[int] = None,
                                       partition_size: int = 0,
                                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attention_decode_scored over an INT8 cache (score forms and masks, no weights)."""
    return prepare_paged_attention_decode_scored_int8(
        q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, out, softcap=softcap, slopes=slopes,
        window=window, starts=starts, max_context_len=max_context_len, partition_size=partition_size,
        workspace=workspace)()


def prepare_paged_attention_decode_scored_int8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                               k_scale: torch.Tensor, v_scale: torch.Tensor,
                                               block_tables: torch.Tensor, context_lens: torch.Tensor,
                                               scale: Optional[float] = None, out: Optional[torch.Tensor] = None, *,
                                               softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                                               window: int = 0, starts: Optional[torch.Tensor] = None,
                                               max_context_len: Optional[int] = None, partition_size: int = 0,
                                               workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """paged_attention_decode_scored_int8, checked and marshalled once (see PreparedCall)."""
    return _prepare_decode_scored("pkv_paged_attention_decode_scored_int8", q, k_cache, v_cache, (k_scale, v_scale),
                                  block_tables, context_lens, scale, out, softcap, slopes, window, starts, None, None,
                                  max_context_len, partition_size, workspace)


def prefill_scored_workspace_bytes(num_rows, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                   max_query_len, max_context_len, window=0, has_prefix=False, kv_splits=0) -> int:
    n = lib().pkv_prefill_scored_workspace_bytes(num_rows, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                 max_query_len, max_context_len, window, int(has_prefix), kv_splits)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError("pkv_prefill_scored_workspace_bytes", 1)
    return int(n)


def paged_attention_prefill_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_tables: torch.Tensor, query_start: torch.Tensor, context_lens: torch.Tensor,
                                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None, *,
                                   max_query_len: int, max_context_len: int, softcap: float = 0.0,
                                   slopes: Optional[torch.Tensor] = None, window: int = 0,
                                   starts: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None,
                                   kv_splits: int = 0, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attention_prefill with capped scores, a distance bias (slopes fp32 [Hq]), and an
    interval of visible tokens per row: the last ``window`` up to the row's position, from
    ``starts`` (int32 [num_rows], the row's document) on, and always the sequence's first
    ``prefix_lens`` (int32 [B]) tokens that the interval reaches; a row that sees nothing
    gets zeros."""
    return prepare_paged_attention_prefill_scored(
        q, k_cache, v_cache, block_tables, query_start, context_lens, scale, out, max_query_len=max_query_len,
        max_context_len=max_context_len, softcap=softcap, slopes=slopes, window=window, starts=starts,
        prefix_lens=prefix_lens, kv_splits=kv_splits, workspace=workspace)()


def prepare_paged_attention_prefill_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                           block_tables: torch.Tensor, query_start: torch.Tensor,
                                           context_lens: torch.Tensor, scale: Optional[float] = None,
                                           out: Optional[torch.Tensor] = None, *, max_query_len: int,
                                           max_context_len: int, softcap: float = 0.0,
                                           slopes: Optional[torch.Tensor] = None, window: int = 0,
                                           starts: Optional[torch.Tensor] = None,
                                           prefix_lens: Optional[torch.Tensor] = None, kv_splits: int = 0,
                                           workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """paged_attention_prefill_scored, checked and marshalled once (see PreparedCall); the
    call returns ``out``.  Without ``workspace`` it holds one of its own."""
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    if q.dim() != 3 or q.shape[2] != d or not q.is_contiguous() or q.dtype != k_cache.dtype:
        raise ValueError(f"q must be a contiguous [num_rows, num_q_heads, {d}] of the cache dtype")
    rows, hq = int(q.shape[0]), int(q.shape[1])
    b = int(context_lens.numel())
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b \
            or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks_per_seq]")
    if query_start.dtype != torch.int32 or query_start.numel() != b + 1 or not query_start.is_contiguous():
        raise ValueError("query_start must be a contiguous int32 [num_seqs + 1]")
    if context_lens.dtype != torch.int32 or not context_lens.is_contiguous():
        raise ValueError("context_lens must be a contiguous int32 [num_seqs]")
    _check_scores(softcap, slopes, window, hq)
    _int32(window=window, kv_splits=kv_splits, max_query_len=max_query_len, max_context_len=max_context_len)
    for name, t, n in (("starts", starts, rows), ("prefix_lens", prefix_lens, b)):
        if t is not None and (t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 [{n}]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must match q")
    _one_device(q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables, query_start=query_start,
                context_lens=context_lens, out=out, slopes=slopes, starts=starts, prefix_lens=prefix_lens)
    with torch.cuda.device(q.device):
        need = prefill_scored_workspace_bytes(rows, b, hq, hkv, d, bs, max_query_len, max_context_len, window,
                                              prefix_lens is not None, kv_splits)
    workspace = _own_workspace(q.device, need, workspace)
    ptr = lambda t: None if t is None else t.data_ptr()
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), nb, stride, block_tables.data_ptr(),
            int(block_tables.shape[1]), query_start.data_ptr(), context_lens.data_ptr(), rows, int(max_query_len),
            int(max_context_len), b, hq, hkv, d, bs, float(scale), float(softcap), ptr(slopes), int(window),
            ptr(starts), ptr(prefix_lens), out.data_ptr(), ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(), int(kv_splits), _dtype_code(q))
    return PreparedCall("pkv_paged_attention_prefill_scored", args, q.device,
                        (q, k_cache, v_cache, block_tables, query_start, context_lens, out, slopes, starts,
                         prefix_lens, workspace), out)


# ---------------------------------------------------------------------------
# Eviction by accumulated attention weight
# ---------------------------------------------------------------------------

def evict_select(weights: torch.Tensor, context_lens: torch.Tensor, budget: int, *, sinks: int = 0, recent: int = 0,
                 max_context_len: Optional[int] = None, weights_out: Optional[torch.Tensor] = None,
                 kept: Optional[torch.Tensor] = None,
                 kept_lens: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Which tokens of each (sequence, KV head) stay: (kept int32 [B, Hkv, budget] ascending
    positions then -1, kept_lens int32 [B] = min(length, budget)).

    A longer context keeps its first ``sinks``, its last ``recent`` and the heaviest of
    the tokens between (equal weights: the lower position).  weights: fp32 [B, Hkv, W],
    W >= max_context_len, as paged_attention_decode_scored accumulates them;
    ``weights_out`` (may be ``weights``) gets the kept weights in their new places and
    zeros up to the old length.  ``kept_lens`` must not be ``context_lens``: evict_compact
    needs both."""
    return prepare_evict_select(weights, context_lens, budget, sinks=sinks, recent=recent,
                                max_context_len=max_context_len, weights_out=weights_out, kept=kept,
                                kept_lens=kept_lens)()


def prepare_evict_select(weights: torch.Tensor, context_lens: torch.Tensor, budget: int, *, sinks: int = 0,
                         recent: int = 0, max_context_len: Optional[int] = None,
                         weights_out: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
                         kept_lens: Optional[torch.Tensor] = None) -> PreparedCall:
    """evict_select, checked and marshalled once (see PreparedCall); the call returns
    (kept, kept_lens)."""
    if weights.dtype != torch.float32 or weights.dim() != 3 or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous float32 [num_seqs, num_kv_heads, max_tokens]")
    b, hkv, width = (int(x) for x in weights.shape)
    if context_lens.dtype != torch.int32 or context_lens.numel() != b or not context_lens.is_contiguous():
        raise ValueError("context_lens must be a contiguous int32 [num_seqs]")
    if weights_out is not None and (weights_out.dtype != torch.float32 or weights_out.shape != weights.shape
                                    or not weights_out.is_contiguous()):
        raise ValueError("weights_out must match weights")
    _int32(budget=budget, max_context_len=max_context_len or 0)
    if budget <= 0 or sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("budget must be positive and cover sinks + recent")
    if max_context_len is None:
        max_context_len = int(context_lens.max().item()) if b else 0
    if max_context_len > width:
        raise ValueError("weights must have a column for every context token")
    if kept is None:
        kept = torch.empty((b, hkv, budget), dtype=torch.int32, device=weights.device)
    elif kept.dtype != torch.int32 or kept.shape != (b, hkv, budget) or not kept.is_contiguous():
        raise ValueError("kept must be a contiguous int32 [num_seqs, num_kv_heads, budget]")
    if kept_lens is None:
        kept_lens = torch.empty(b, dtype=torch.int32, device=weights.device)
    elif kept_lens.dtype != torch.int32 or kept_lens.numel() != b or not kept_lens.is_contiguous():
        raise ValueError("kept_lens must be a contiguous int32 [num_seqs]")
    if abs(kept_lens.data_ptr() - context_lens.data_ptr()) < 4 * b:
        raise ValueError("kept_lens must not overlap context_lens")
    _one_device(weights, context_lens=context_lens, weights_out=weights_out, kept=kept, kept_lens=kept_lens)
    args = (weights.data_ptr(), width, context_lens.data_ptr(), int(max_context_len), b, hkv, int(budget), int(sinks),
            int(recent), None if weights_out is None else weights_out.data_ptr(), kept.data_ptr(),
            kept_lens.data_ptr())
    return PreparedCall("pkv_evict_select", args, weights.device, (weights, context_lens, weights_out, kept, kept_lens),
                        (kept, kept_lens))


def evict_compact(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, kept: torch.Tensor, kept_lens: torch.Tensor, *,
                  dst_block_tables: Optional[torch.Tensor] = None) -> None:
    """Move the K and V rows of the kept tokens (evict_select) to the front of each
    sequence's context: into the fresh blocks of ``dst_block_tables``, or in place (the
    blocks that get rows must belong to their sequence alone: BlockManager.make_private).
    Afterwards kept_lens are the context lengths."""
    prepare_evict_compact(k_cache, v_cache, block_tables, context_lens, kept, kept_lens,
                          dst_block_tables=dst_block_tables)()


def prepare_evict_compact(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                          context_lens: torch.Tensor, kept: torch.Tensor, kept_lens: torch.Tensor, *,
                          dst_block_tables: Optional[torch.Tensor] = None) -> PreparedCall:
    """evict_compact, checked and marshalled once (see PreparedCall)."""
    nb, hkv, bs, d, stride = _cache_geometry(k_cache, v_cache)
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks_per_seq]")
    b = int(block_tables.shape[0])
    for name, t in (("context_lens", context_lens), ("kept_lens", kept_lens)):
        if t.dtype != torch.int32 or t.numel() != b or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 [num_seqs]")
    if kept.dtype != torch.int32 or kept.dim() != 3 or tuple(kept.shape[:2]) != (b, hkv) or not kept.is_contiguous():
        raise ValueError("kept must be a contiguous int32 [num_seqs, num_kv_heads, budget]")
    if dst_block_tables is not None and (dst_block_tables.dtype != torch.int32 or dst_block_tables.dim() != 2
                                         or dst_block_tables.shape[0] != b or not dst_block_tables.is_contiguous()):
        raise ValueError("dst_block_tables must be a contiguous int32 [num_seqs, blocks]")
    _one_device(k_cache, v_cache=v_cache, block_tables=block_tables, context_lens=context_lens, kept=kept,
                kept_lens=kept_lens, dst_block_tables=dst_block_tables)
    dst = dst_block_tables
    args = (k_cache.data_ptr(), v_cache.data_ptr(), nb, stride, hkv, d, bs, block_tables.data_ptr(),
            int(block_tables.shape[1]), context_lens.data_ptr(), b, kept.data_ptr(), kept_lens.data_ptr(),
            int(kept.shape[2]), None if dst is None else dst.data_ptr(), 0 if dst is None else int(dst.shape[1]),
            _cache_dtype_code(k_cache))
    return PreparedCall("pkv_evict_compact", args, k_cache.device,
                        (k_cache, v_cache, block_tables, context_lens, kept, kept_lens, dst))


def get_device_error(device: Optional[torch.device] = None) -> Tuple[int, list]:
    """Synchronise, read and clear the device status word: (flags, [names])."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    flags = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        st = lib().pkv_get_device_error(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream),
                                        ctypes.byref(flags))
    if st not in (0, 4):
        raise PagedKVError("pkv_get_device_error", st)
    names = [n for bit, n in DEVERR.items() if flags.value & bit]
    return int(flags.value), names


def launch_count() -> int:
    return int(lib().pkv_launch_count())


def decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len,
                partition_size, sm_count, int8=False) -> dict:
    """The library's launch decision for these arguments (pure host function): that of
    pkv_paged_attention_decode, or of the INT8-cache decode when ``int8``."""
    outs = [ctypes.c_int(0) for _ in range(4)]
    name = "pkv_decode_int8_plan" if int8 else "pkv_decode_plan"
    st = getattr(lib(), name)(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                              max_context_len, partition_size, sm_count,
                              *[ctypes.byref(o) for o in outs])
    _check(st, name)
    return {"partition_size": outs[0].value, "num_partitions": outs[1].value,
            "heads_per_block": outs[2].value, "needs_merge": bool(outs[3].value)}


def debug_wait_timeout(timeout_ns: int, device: Optional[torch.device] = None) -> None:
    """Launch the bounded-wait self test (see pkv_debug_wait_timeout)."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    with torch.cuda.device(dev):
        st = lib().pkv_debug_wait_timeout(int(timeout_ns),
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    _check(st, "pkv_debug_wait_timeout")
