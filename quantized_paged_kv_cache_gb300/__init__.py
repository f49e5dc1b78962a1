"""Paged INT8 group-64 KV cache for one GB300: append, split-KV decode attention, combine.

The functions below mirror the C ABI in ``include/nk.h`` one to one and take
torch tensors that already live on the GPU. They only marshal arguments: the
work runs in the library's CUDA kernels on the current CUDA stream. Nothing
here synchronizes; errors in device data are reported through the optional
int32 ``status`` tensor (``NK_DEVFLAG_*`` bits).
"""
from __future__ import annotations

import ctypes
import functools
import numbers
from dataclasses import dataclass

from ._lib import NKError, lib, nk_kv_pool, status_string  # noqa: F401

NK_DEVFLAG_BAD_PAGE = 0x1
NK_DEVFLAG_BAD_POS = 0x2
NK_DEVFLAG_BAD_CTX = 0x4
NK_DEVFLAG_TIMEOUT = 0x8
NK_DEVFLAG_RANGE = 0x10
NK_DEVFLAG_NO_PAGES = 0x20
NK_DEVFLAG_BAD_TOKEN = 0x40
GROUP = 64
MAX_T = 16

__all__ = [
    "KVPool", "NKError", "kv_chunk_bytes", "kv_pool_bytes", "kv_append", "decode_default_splits", "decode_default_ctas",
    "decode_workspace_bytes", "paged_decode_attn", "paged_decode_attn_simt", "paged_decode_attn_noalloc",
    "attn_combine", "status_string", "decode_step", "rk8v4_chunk_bytes", "rk8v4_pool_bytes", "rk8v4_append",
    "rk8v4_decode_attn", "i8f16_chunk_bytes", "i8f16_pool_bytes", "i8f16_append", "i8f16_decode_attn",
    "bf16kv_chunk_bytes", "bf16kv_pool_bytes", "bf16kv_append", "bf16kv_decode_attn", "test_inject_copy_stall", "paged_prefill_attn",
    "step_tables", "mrope", "paged_window_attn", "chunk_workspace_bytes", "paged_chunk_attn",
    "PageBounds", "page_bounds_bytes", "page_bounds", "page_select_workspace_bytes", "page_select", "paged_sparse_attn",
    "page_weights_workspace_bytes", "page_weights", "evict_pages", "verify_drafts",
]


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _raw_stream():
    """torch's call for the current stream's handle, without the Stream object
    around it (2.9 us of a call's host time on a Grace core, against 0.2)."""
    import torch

    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


_current = None


def _stream(stream) -> int:
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    global _current
    if _current is None:
        import torch

        torch.cuda.current_stream()  # CUDA is up before the raw handle is asked for
        _current = _raw_stream()
    return _current()


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise NKError(rc, where)


def _need_cuda(*tensors) -> None:
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def kv_chunk_bytes(page_size: int, head_dim: int) -> int:
    return int(lib().nk_kv_chunk_bytes(page_size, head_dim))


def kv_pool_bytes(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().nk_kv_pool_bytes(num_pages, page_size, num_kv_heads, head_dim))


def i8f16_chunk_bytes(page_size: int, head_dim: int) -> int:
    return int(lib().nk_i8f16_chunk_bytes(page_size, head_dim))


def i8f16_pool_bytes(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().nk_i8f16_pool_bytes(num_pages, page_size, num_kv_heads, head_dim))


def bf16kv_chunk_bytes(page_size: int, head_dim: int) -> int:
    return int(lib().nk_bf16kv_chunk_bytes(page_size, head_dim))


def bf16kv_pool_bytes(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().nk_bf16kv_pool_bytes(num_pages, page_size, num_kv_heads, head_dim))


def rk8v4_chunk_bytes(page_size: int, head_dim: int) -> int:
    return int(lib().nk_rk8v4_chunk_bytes(page_size, head_dim))


def rk8v4_pool_bytes(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().nk_rk8v4_pool_bytes(num_pages, page_size, num_kv_heads, head_dim))


@dataclass
class KVPool:
    """A caller-owned pool: ``storage`` is a uint8 CUDA tensor laid out as
    [page][kv-head][chunk], in the INT8 group-64 format with fp32 scales
    (``fmt="int8"``, ``kv_pool_bytes(...)`` bytes), the rk8v4 format
    (``"rk8v4"``), the pages' INT8 layout with fp16 scales (``"i8f16"``) or
    bf16 rows (``"bf16"``), each sized by its own ``*_pool_bytes``."""

    storage: "object"
    num_pages: int
    page_size: int
    num_kv_heads: int
    head_dim: int
    fmt: str = "int8"

    @classmethod
    def empty(cls, num_pages, page_size, num_kv_heads, head_dim, device="cuda", fill: int | None = None,
              fmt: str = "int8"):
        import torch

        sizers = {"int8": kv_pool_bytes, "rk8v4": rk8v4_pool_bytes, "i8f16": i8f16_pool_bytes,
                  "bf16": bf16kv_pool_bytes}
        if fmt not in sizers:
            raise ValueError(f"unknown KV format {fmt!r}")
        n = sizers[fmt](num_pages, page_size, num_kv_heads, head_dim)
        st = torch.empty(n, dtype=torch.uint8, device=device)
        if fill is not None:
            st.fill_(fill)
        return cls(st, num_pages, page_size, num_kv_heads, head_dim, fmt)

    def need(self, fmt: str) -> None:
        if self.fmt != fmt:
            raise ValueError(f"this call needs a {fmt} pool, not a {self.fmt} one")

    def c_struct(self) -> nk_kv_pool:
        _need_cuda(self.storage)
        return self._struct()

    def _struct(self) -> nk_kv_pool:  # (of storage that was checked)
        return nk_kv_pool(self.storage.data_ptr(), self.num_pages, self.page_size, self.num_kv_heads, self.head_dim)


def kv_append(pool: KVPool, block_table, start_pos, cu_new, k, v, status=None, stream=None) -> None:
    """Quantize k/v rows (bf16 [total_new][Hkv][D]) into the pool (nk_kv_append)."""
    _need_cuda(block_table, start_pos, cu_new, k, v, status)
    pool.need("int8")
    B = int(start_pos.numel())
    total = int(k.shape[0]) if k.dim() > 0 else 0
    ps = pool.c_struct()
    rc = lib().nk_kv_append(ctypes.byref(ps), _ptr(block_table), int(block_table.shape[-1]), _ptr(start_pos),
                            _ptr(cu_new), B, total, _ptr(k), _ptr(v), _ptr(status), _stream(stream))
    _check(rc, "nk_kv_append")


def decode_default_splits(B: int, num_kv_heads: int, max_ctx: int, page_size: int) -> int:
    """Default split (CTA) count of the decode calls (nk_decode_default_splits)."""
    return int(lib().nk_decode_default_splits(B, num_kv_heads, max_ctx, page_size))


def decode_default_ctas(B: int, num_kv_heads: int, max_ctx: int, page_size: int) -> int:
    """The same count under its earlier name (nk_decode_default_ctas)."""
    return int(lib().nk_decode_default_ctas(B, num_kv_heads, max_ctx, page_size))


def decode_workspace_bytes(B: int, T: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                           num_ctas: int = 0) -> int:
    return int(lib().nk_decode_workspace_bytes(B, T, num_q_heads, num_kv_heads, head_dim, num_ctas))


def _decode(fn, name, pool, q, block_table, ctx_lens, sm_scale, max_ctx, num_ctas, workspace, out, status, stream,
            fmt="int8"):
    import torch

    _need_cuda(q, block_table, ctx_lens, workspace, out, status)
    pool.need(fmt)
    B, T, Hq, D = (int(s) for s in q.shape)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        nbytes = decode_workspace_bytes(B, T, Hq, pool.num_kv_heads, D, num_ctas)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    ps = pool.c_struct()
    wbytes = workspace.numel() * workspace.element_size()
    rc = fn(ctypes.byref(ps), _ptr(q), _ptr(block_table), int(block_table.shape[-1]), _ptr(ctx_lens), B, T, Hq,
            float(sm_scale), int(max_ctx), int(num_ctas), _ptr(workspace), wbytes, _ptr(out), _ptr(status),
            _stream(stream))
    _check(rc, name)
    return out


def paged_decode_attn(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int, num_ctas: int = 0,
                      workspace=None, out=None, status=None, stream=None):
    """Split-KV paged attention on tensor cores (nk_paged_decode_attn); returns out bf16 [B][T][Hq][D]."""
    return _decode(lib().nk_paged_decode_attn, "nk_paged_decode_attn", pool, q, block_table, ctx_lens, sm_scale,
                   max_ctx, num_ctas, workspace, out, status, stream)


def paged_decode_attn_simt(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int,
                           num_ctas: int = 0, workspace=None, out=None, status=None, stream=None):
    """Same result from the fp32 CUDA-core kernel (nk_paged_decode_attn_simt)."""
    return _decode(lib().nk_paged_decode_attn_simt, "nk_paged_decode_attn_simt", pool, q, block_table, ctx_lens,
                   sm_scale, max_ctx, num_ctas, workspace, out, status, stream)


def decode_step(pool: KVPool, block_table, start_pos, cu_new, k, v, q, ctx_lens, sm_scale: float, max_ctx: int,
                num_ctas: int = 0, workspace=None, out=None, status=None, stream=None):
    """kv_append of the step's rows, then paged_decode_attn, in one call
    (nk_decode_step); returns out bf16 [B][T][Hq][D]."""
    import torch

    _need_cuda(block_table, start_pos, cu_new, k, v, q, ctx_lens, workspace, out, status)
    pool.need("int8")
    B, T, Hq, D = (int(s) for s in q.shape)
    if int(start_pos.numel()) != B:
        raise ValueError("start_pos must hold one position per sequence of q")
    total = int(k.shape[0]) if k.dim() > 0 else 0
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        nbytes = decode_workspace_bytes(B, T, Hq, pool.num_kv_heads, D, num_ctas)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    ps = pool.c_struct()
    wbytes = workspace.numel() * workspace.element_size()
    rc = lib().nk_decode_step(ctypes.byref(ps), _ptr(block_table), int(block_table.shape[-1]), _ptr(start_pos),
                              _ptr(cu_new), total, _ptr(k), _ptr(v), _ptr(q), _ptr(ctx_lens), B, T, Hq,
                              float(sm_scale), int(max_ctx), int(num_ctas), _ptr(workspace), wbytes, _ptr(out),
                              _ptr(status), _stream(stream))
    _check(rc, "nk_decode_step")
    return out


def step_host_layout(B: int, total_new: int, T: int, num_q_heads: int, num_kv_heads: int, head_dim: int):
    """(total bytes, offsets of k, v, q, start_pos, cu_new, ctx_lens) of
    decode_step_host's input buffer (nk_step_host_layout)."""
    offs = (ctypes.c_size_t * 6)()
    total = lib().nk_step_host_layout(int(B), int(total_new), int(T), int(num_q_heads), int(num_kv_heads),
                                      int(head_dim), offs)
    if total == 0:
        raise ValueError("invalid shape for the host step layout")
    return int(total), tuple(int(o) for o in offs)


def decode_step_host(pool: KVPool, block_table, B: int, total_new: int, T: int, num_q_heads: int, sm_scale: float,
                     max_ctx: int, in_host, staging, out, out_host, num_ctas: int = 0, workspace=None, status=None,
                     status_host=None, stream=None):
    """nk_decode_step_host: one step from host memory. in_host is a host
    uint8 tensor (pinned for an asynchronous transfer) in the
    step_host_layout layout; staging a device buffer of at least that size;
    out the device output [B][T][Hq][D] bf16 and out_host its host copy;
    status_host an int32 host tensor of one element. Waits for the stream."""
    import torch

    _need_cuda(block_table, staging, out, workspace, status)
    pool.need("int8")
    if in_host.is_cuda or out_host.is_cuda or (status_host is not None and status_host.is_cuda):
        raise ValueError("in_host, out_host and status_host must be host tensors")
    D = pool.head_dim
    if workspace is None:
        nbytes = decode_workspace_bytes(B, T, num_q_heads, pool.num_kv_heads, D, num_ctas)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=staging.device)
    ps = pool.c_struct()
    wbytes = workspace.numel() * workspace.element_size()
    rc = lib().nk_decode_step_host(ctypes.byref(ps), _ptr(block_table), int(block_table.shape[-1]), int(B),
                                   int(total_new), int(T), int(num_q_heads), float(sm_scale), int(max_ctx),
                                   int(num_ctas), _ptr(in_host), _ptr(staging), _ptr(workspace), wbytes, _ptr(out),
                                   _ptr(out_host), _ptr(status), _ptr(status_host), _stream(stream))
    _check(rc, "nk_decode_step_host")
    return out_host


NOALLOC_MAX_WORKSPACE = 8 << 20


def paged_decode_attn_noalloc(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int,
                              num_ctas: int = 0, out=None, status=None, stream=None):
    """nk_paged_decode_attn_noalloc: the tensor-core decode with its split
    partials in the library's own fixed device array, for callers that cannot
    allocate device memory. Calls that overlap on the GPU race on that array."""
    import torch

    _need_cuda(q, block_table, ctx_lens, out, status)
    pool.need("int8")
    B, T, Hq, D = (int(s) for s in q.shape)
    if out is None:
        out = torch.empty_like(q)
    ps = pool.c_struct()
    rc = lib().nk_paged_decode_attn_noalloc(ctypes.byref(ps), _ptr(q), _ptr(block_table), int(block_table.shape[-1]),
                                            _ptr(ctx_lens), B, T, Hq, float(sm_scale), int(max_ctx), int(num_ctas),
                                            _ptr(out), _ptr(status), _stream(stream))
    _check(rc, "nk_paged_decode_attn_noalloc")
    return out


def rk8v4_append(pool: KVPool, block_table, start_pos, cu_new, k, v, status=None, stream=None) -> None:
    """Rotate, quantize and scatter k/v rows (bf16 [total_new][Hkv][D]) into an rk8v4 pool (nk_rk8v4_append)."""
    _need_cuda(block_table, start_pos, cu_new, k, v, status)
    pool.need("rk8v4")
    B = int(start_pos.numel())
    total = int(k.shape[0]) if k.dim() > 0 else 0
    ps = pool.c_struct()
    rc = lib().nk_rk8v4_append(ctypes.byref(ps), _ptr(block_table), int(block_table.shape[-1]), _ptr(start_pos),
                               _ptr(cu_new), B, total, _ptr(k), _ptr(v), _ptr(status), _stream(stream))
    _check(rc, "nk_rk8v4_append")


def rk8v4_decode_attn(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int, num_ctas: int = 0,
                      workspace=None, out=None, status=None, stream=None):
    """Split-KV paged attention over an rk8v4 pool (nk_rk8v4_decode_attn); returns out bf16 [B][T][Hq][D]."""
    return _decode(lib().nk_rk8v4_decode_attn, "nk_rk8v4_decode_attn", pool, q, block_table, ctx_lens, sm_scale,
                   max_ctx, num_ctas, workspace, out, status, stream, fmt="rk8v4")


def attn_combine(part_o, part_lse, out=None, stream=None):
    """LSE merge of partials: part_o fp32 [S][R][D], part_lse fp32 [S][R] -> bf16 [R][D] (nk_attn_combine)."""
    import torch

    _need_cuda(part_o, part_lse, out)
    S, R, D = (int(s) for s in part_o.shape)
    if out is None:
        out = torch.empty((R, D), dtype=torch.bfloat16, device=part_o.device)
    rc = lib().nk_attn_combine(_ptr(part_o), _ptr(part_lse), S, R, D, _ptr(out), _stream(stream))
    _check(rc, "nk_attn_combine")
    return out


def test_inject_copy_stall(withheld_page: int, wait_cycles: int = 0) -> None:
    """nk_test_inject_copy_stall: failure injection for the bounded-wait tests
    (withheld_page < 0 switches it off)."""
    lib().nk_test_inject_copy_stall(int(withheld_page), int(wait_cycles))


def _fmt_append(fn, name, fmt, pool, block_table, start_pos, cu_new, k, v, status, stream):
    _need_cuda(block_table, start_pos, cu_new, k, v, status)
    pool.need(fmt)
    B = int(start_pos.numel())
    total = int(k.shape[0]) if k.dim() > 0 else 0
    ps = pool.c_struct()
    rc = fn(ctypes.byref(ps), _ptr(block_table), int(block_table.shape[-1]), _ptr(start_pos), _ptr(cu_new), B, total,
            _ptr(k), _ptr(v), _ptr(status), _stream(stream))
    _check(rc, name)


def i8f16_append(pool: KVPool, block_table, start_pos, cu_new, k, v, status=None, stream=None) -> None:
    """Quantize k/v rows into a pool of the pages' INT8 layout with fp16 scales (nk_i8f16_append)."""
    _fmt_append(lib().nk_i8f16_append, "nk_i8f16_append", "i8f16", pool, block_table, start_pos, cu_new, k, v,
                status, stream)


def bf16kv_append(pool: KVPool, block_table, start_pos, cu_new, k, v, status=None, stream=None) -> None:
    """Scatter bf16 k/v rows into a bf16 pool (nk_bf16kv_append)."""
    _fmt_append(lib().nk_bf16kv_append, "nk_bf16kv_append", "bf16", pool, block_table, start_pos, cu_new, k, v,
                status, stream)


def i8f16_decode_attn(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int, num_ctas: int = 0,
                      workspace=None, out=None, status=None, stream=None):
    """Split-KV paged attention over an INT8 pool with fp16 scales (nk_i8f16_decode_attn)."""
    return _decode(lib().nk_i8f16_decode_attn, "nk_i8f16_decode_attn", pool, q, block_table, ctx_lens, sm_scale,
                   max_ctx, num_ctas, workspace, out, status, stream, fmt="i8f16")


def bf16kv_decode_attn(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int, num_ctas: int = 0,
                       workspace=None, out=None, status=None, stream=None):
    """Split-KV paged attention over a bf16 pool (nk_bf16kv_decode_attn)."""
    return _decode(lib().nk_bf16kv_decode_attn, "nk_bf16kv_decode_attn", pool, q, block_table, ctx_lens, sm_scale,
                   max_ctx, num_ctas, workspace, out, status, stream, fmt="bf16")


def paged_prefill_attn(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int, out=None, status=None,
                       stream=None):
    """Chunked-prefill attention of T query tokens per sequence over the paged
    INT8 cache (nk_paged_prefill_attn); returns out bf16 [B][T][Hq][D]."""
    import torch

    _need_cuda(q, block_table, ctx_lens, out, status)
    pool.need("int8")
    B, T, Hq, D = (int(x) for x in q.shape)
    if out is None:
        out = torch.empty_like(q)
    ps = pool.c_struct()
    rc = lib().nk_paged_prefill_attn(ctypes.byref(ps), _ptr(q), _ptr(block_table), int(block_table.shape[-1]),
                                     _ptr(ctx_lens), B, T, Hq, float(sm_scale), int(max_ctx), _ptr(out), _ptr(status),
                                     _stream(stream))
    _check(rc, "nk_paged_prefill_attn")
    return out


_I32_MAX = 2**31 - 1


_device = None


def _here() -> int:
    """Index of the device that launches go to (-2 without a GPU: no tensor lies there)."""
    global _device
    if _device is None:
        import torch

        if not torch.cuda.is_available():
            return -2
        _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        torch.cuda.current_device()  # CUDA is up before the raw call
    return _device()


def _refuse(t, here: int, dtype=None) -> None:
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
    if t.get_device() != here:
        raise ValueError(f"a tensor lies on {t.device}, the call runs on the current device, cuda:{here}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"expected a {dtype} tensor, not a {t.dtype} one")
    raise ValueError("all tensors must be contiguous")


def _need(dtype, *tensors) -> None:
    """On the current device, where the kernels run, contiguous and of one type (None: an argument that is not given)."""
    here = _here()
    for t in tensors:
        if t is not None and not (t.get_device() == here and t.dtype == dtype and t.is_contiguous()):
            _refuse(t, here, dtype)


def _need_scratch(storage, workspace) -> None:
    """The pool's memory and the workspace: of any type."""
    here = _here()
    if not (storage.get_device() == here and storage.is_contiguous()):
        _refuse(storage, here)
    if workspace is not None and not (workspace.get_device() == here and workspace.is_contiguous()):
        _refuse(workspace, here)


def _one(t, what: str) -> None:
    if t.numel() < 1:
        raise ValueError(f"{what} must hold an entry")


def _clamped(max_ctx: int, window: int, sinks: int) -> tuple:
    """A window or sinks past 2^31 - 1 tokens, which the C calls cannot take, mean the same as that many; negative ones
    stay negative, which the C calls refuse."""
    if not -_I32_MAX <= max_ctx <= _I32_MAX:
        raise ValueError("max_ctx must be below 2^31")
    return max(min(window, _I32_MAX), -1), max(min(sinks, _I32_MAX), -1)


def _empty(stream, like, shape, dtype=None):
    """A call's own output or workspace, allocated on the stream the call runs
    on: memory of another stream could still be in use there, or be handed out
    again while the call uses it."""
    import torch

    if stream is None:  # (rows of consecutive heads: dense ones, whatever the rows of `like` are apart)
        return torch.empty_like(like) if dtype is None else torch.empty(shape, dtype=dtype, device=like.device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = _stream(stream)
        stream = torch.cuda.ExternalStream(raw, device=like.device) if raw else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)


def step_tables(page_size: int, num_pages: int, start_pos, new_lens, free_pages, block_table, cu_new, ctx_lens, slot_map,
                positions=None, used=None, status=None, stream=None) -> None:
    """The block tables, slot map and lengths of a step from its requests'
    lengths and a list of free pages (nk_step_tables): ``block_table`` int32
    [B][max_pages] is updated in place; ``cu_new`` int32 [B+1], ``ctx_lens``
    int32 [B], ``slot_map`` int64 [max_rows], ``positions`` int32 [max_rows]
    and ``used`` int32 [1] are written."""
    import torch

    _need(torch.int32, start_pos, new_lens, free_pages, block_table, cu_new, ctx_lens, positions, used, status)
    _need(torch.int64, slot_map)
    if used is not None:
        _one(used, "used")
    if page_size > _I32_MAX or num_pages > _I32_MAX or page_size < -_I32_MAX or num_pages < -_I32_MAX:
        raise ValueError("page_size and num_pages must be below 2^31")
    B, rows, shape = start_pos.numel(), min(slot_map.numel(), _I32_MAX), block_table.shape
    if new_lens.numel() != B or ctx_lens.numel() != B or cu_new.numel() != B + 1 or len(shape) != 2 or shape[0] != B:
        raise ValueError("start_pos, new_lens, ctx_lens and block_table hold one entry (row) per sequence, cu_new one more")
    if positions is not None and positions.numel() < rows:
        raise ValueError("positions must hold an entry for every one of slot_map")
    rc = lib().nk_step_tables(page_size, num_pages, start_pos.data_ptr(), new_lens.data_ptr(), B, free_pages.data_ptr(),
                              min(free_pages.numel(), _I32_MAX), block_table.data_ptr(), shape[1], cu_new.data_ptr(),
                              ctx_lens.data_ptr(), slot_map.data_ptr(), _ptr(positions), rows, _ptr(used), _ptr(status),
                              _stream(stream))
    _check(rc, "nk_step_tables")


@functools.lru_cache(maxsize=64)
def _sections(sections: tuple):
    """(the sections as a C array, its address, their count, their sum); the array is only ever read."""
    if not all(isinstance(x, numbers.Integral) for x in sections):
        raise ValueError("sections must be whole numbers")
    array = (ctypes.c_int32 * len(sections))(*map(int, sections))
    return array, ctypes.addressof(array), len(sections), sum(sections)


def _row_stride(t, shape, what: str) -> int:
    """Row stride of [rows][heads][head_dim] rows whose heads are consecutive."""
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise ValueError(f"the heads of a row of {what} must be consecutive")
    return s0 if n > 1 else h * d


def mrope(q, k, positions, inv_freq, sections, interleaved: bool = False, q_out=None, k_out=None, num_rows=None,
          stream=None):
    """Rotary positions with several axes on query and key rows (nk_mrope):
    ``q`` bf16 [rows][Hq][D] and ``k`` [rows][Hkv][D] (rows may be strided),
    ``positions`` int32 [axes][rows], ``inv_freq`` float64 [half] on the host,
    ``sections`` the frequencies of each axis. Returns (q_out, k_out); pass
    q and k themselves to rotate in place."""
    import torch

    qs, ks, ps = q.shape, k.shape, positions.shape
    if len(qs) != 3 or len(ks) != 3 or ks[0] != qs[0] or ks[2] != qs[2]:
        raise ValueError("q and k must be [rows][heads][head_dim] with the same rows and head_dim")
    _need(torch.int32, positions, num_rows)
    bf16, here = torch.bfloat16, _here()
    for t in (q, k, q_out, k_out):
        if t is not None and not (t.get_device() == here and t.dtype == bf16):
            _refuse(t, here, bf16)
    if inv_freq.is_cuda or inv_freq.dtype != torch.float64 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 host tensor")
    if num_rows is not None:
        _one(num_rows, "num_rows")
    _, array, axes, half = _sections(tuple(sections))
    rows, Hq, D = qs
    if rows > _I32_MAX:
        raise ValueError("q and k must have fewer than 2^31 rows")
    Hkv = ks[1]
    if len(ps) != 2 or ps[0] != axes or ps[1] < rows:
        raise ValueError("positions must hold one row of positions per section (axis)")
    if inv_freq.numel() != half:
        raise ValueError("inv_freq must hold one frequency for every one of the sections")
    if q_out is None:
        q_out, qos = _empty(stream, q, qs), Hq * D
    elif q_out.shape == qs:
        qos = _row_stride(q_out, qs, "q_out")
    else:
        raise ValueError("q_out must have the shape of q")
    if k_out is None:
        k_out, kos = _empty(stream, k, ks), Hkv * D
    elif k_out.shape == ks:
        kos = _row_stride(k_out, ks, "k_out")
    else:
        raise ValueError("k_out must have the shape of k")
    rc = lib().nk_mrope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), _row_stride(q, qs, "q"),
                        _row_stride(k, ks, "k"), qos, kos, rows, Hq, Hkv, D, positions.data_ptr(), ps[1],
                        inv_freq.data_ptr(), array, axes, 1 if interleaved else 0, _ptr(num_rows), _stream(stream))
    _check(rc, "nk_mrope")
    return q_out, k_out


def paged_window_attn(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int, window: int,
                      sinks: int = 0, num_ctas: int = 0, workspace=None, out=None, status=None, stream=None):
    """Decode / verify attention over a sliding window and the first ``sinks``
    tokens (nk_paged_window_attn); returns out bf16 [B][T][Hq][D]."""
    import torch

    _need(torch.bfloat16, q, out)
    _need(torch.int32, block_table, ctx_lens, status)
    _need_scratch(pool.storage, workspace)
    pool.need("int8")
    if not (0 <= max_ctx <= _I32_MAX and 0 <= window <= _I32_MAX and 0 <= sinks <= _I32_MAX):
        window, sinks = _clamped(max_ctx, window, sinks)
    B, T, Hq, D = q.shape
    shape = block_table.shape
    if D != pool.head_dim or len(shape) != 2 or shape[0] != B or ctx_lens.numel() != B:
        raise ValueError("q, block_table, ctx_lens and the pool disagree on the batch or the head dim")
    if out is None:
        out = _empty(stream, q, q.shape)
    elif out.numel() != q.numel():
        raise ValueError("out must have the shape of q")
    if workspace is None:
        wbytes = max(lib().nk_decode_workspace_bytes(B, T, Hq, pool.num_kv_heads, D, num_ctas), 256)
        workspace = _empty(stream, q, wbytes, torch.uint8)
    else:
        wbytes = workspace.numel() * workspace.element_size()
    rc = lib().nk_paged_window_attn(pool._struct(), q.data_ptr(), block_table.data_ptr(), shape[1],
                                    ctx_lens.data_ptr(), B, T, Hq, sm_scale, max_ctx, window, sinks, num_ctas,
                                    workspace.data_ptr(), wbytes, out.data_ptr(), _ptr(status), _stream(stream))
    _check(rc, "nk_paged_window_attn")
    return out


def chunk_workspace_bytes(head_dim: int, num_ctas: int = 0) -> int:
    return int(lib().nk_chunk_workspace_bytes(head_dim, num_ctas))


def paged_chunk_attn(pool: KVPool, q, cu_q, block_table, ctx_lens, sm_scale: float, max_ctx: int, window: int = 0,
                     sinks: int = 0, num_ctas: int = 0, workspace=None, out=None, status=None, stream=None):
    """Attention of ragged chunks of new tokens over the paged cache
    (nk_paged_chunk_attn): ``q`` bf16 [total_q][Hq][D], the rows of sequence b
    at cu_q[b] .. cu_q[b+1]-1; returns out bf16 [total_q][Hq][D]."""
    import torch

    _need(torch.bfloat16, q, out)
    _need(torch.int32, cu_q, block_table, ctx_lens, status)
    _need_scratch(pool.storage, workspace)
    pool.need("int8")
    if not (0 <= max_ctx <= _I32_MAX and 0 <= window <= _I32_MAX and 0 <= sinks <= _I32_MAX):
        window, sinks = _clamped(max_ctx, window, sinks)
    total, Hq, D = q.shape
    B, shape = ctx_lens.numel(), block_table.shape
    if D != pool.head_dim or len(shape) != 2 or shape[0] != B or cu_q.numel() != B + 1:
        raise ValueError("q, cu_q, block_table, ctx_lens and the pool disagree on the batch or the head dim")
    if out is None:
        out = _empty(stream, q, q.shape)
    elif out.numel() != q.numel():
        raise ValueError("out must have the shape of q")
    if workspace is None:
        wbytes = lib().nk_chunk_workspace_bytes(D, num_ctas)
        workspace = _empty(stream, q, wbytes, torch.uint8)
    else:
        wbytes = workspace.numel() * workspace.element_size()
    rc = lib().nk_paged_chunk_attn(pool._struct(), q.data_ptr(), cu_q.data_ptr(), block_table.data_ptr(), shape[1],
                                   ctx_lens.data_ptr(), B, total, Hq, sm_scale, max_ctx, window, sinks, num_ctas,
                                   workspace.data_ptr(), wbytes, out.data_ptr(), _ptr(status), _stream(stream))
    _check(rc, "nk_paged_chunk_attn")
    return out


def page_bounds_bytes(num_pages: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().nk_page_bounds_bytes(num_pages, num_kv_heads, head_dim))


@dataclass
class PageBounds:
    """The caller-owned bounds of a pool's keys: ``storage`` is a uint8 CUDA
    tensor of ``page_bounds_bytes(...)`` bytes, codes [page][kv-head][hi, lo][D]
    int8 followed by scales [page][kv-head] fp32 (nk_page_bounds)."""

    storage: "object"
    num_pages: int
    num_kv_heads: int
    head_dim: int

    @classmethod
    def empty(cls, pool: KVPool):
        """Bounds for ``pool``, all zeros."""
        import torch

        n = page_bounds_bytes(pool.num_pages, pool.num_kv_heads, pool.head_dim)
        return cls(torch.zeros(n, dtype=torch.uint8, device=pool.storage.device), pool.num_pages, pool.num_kv_heads,
                   pool.head_dim)

    def _codes_bytes(self) -> int:
        return self.num_pages * self.num_kv_heads * 2 * self.head_dim

    def codes(self):
        """int8 [num_pages][Hkv][2][D], a view."""
        import torch

        n = self._codes_bytes()
        return self.storage[:n].view(torch.int8).view(self.num_pages, self.num_kv_heads, 2, self.head_dim)

    def scales(self):
        """fp32 [num_pages][Hkv], a view."""
        import torch

        n = self._codes_bytes()
        return self.storage[n:n + 4 * self.num_pages * self.num_kv_heads].view(torch.float32).view(
            self.num_pages, self.num_kv_heads)

    def values(self, out=None, stream=None):
        """fp32 [num_pages][Hkv][2][D]: the largest and smallest values that the codes stand for (nk_page_bounds_values)."""
        import torch

        _need_scratch(self.storage, None)
        self._check()
        shape = (self.num_pages, self.num_kv_heads, 2, self.head_dim)
        if out is None:
            out = _empty(stream, self.storage, shape, torch.float32)
        else:
            _need(torch.float32, out)
            if out.shape != shape:
                raise ValueError("out must be [num_pages][kv-heads][2][head_dim]")
        rc = lib().nk_page_bounds_values(self.storage.data_ptr(), self.num_pages, self.num_kv_heads, self.head_dim,
                                         out.data_ptr(), _stream(stream))
        _check(rc, "nk_page_bounds_values")
        return out

    def _check(self) -> None:
        storage = self.storage
        if storage.element_size() != 1 or storage.numel() < self.num_pages * self.num_kv_heads * (2 * self.head_dim + 4):
            raise ValueError("the bounds' storage must be a tensor of page_bounds_bytes(...) bytes")


def page_bounds(pool: KVPool, bounds: PageBounds, block_table, start_pos, cu_new, status=None, stream=None) -> None:
    """The bounds of the pages that a step's new rows fall in, after their
    kv_append (nk_page_bounds); block_table, start_pos and cu_new as there."""
    import torch

    _need(torch.int32, block_table, start_pos, cu_new, status)
    _need_scratch(pool.storage, bounds.storage)
    pool.need("int8")
    bounds._check()
    if (bounds.num_pages, bounds.num_kv_heads, bounds.head_dim) != (pool.num_pages, pool.num_kv_heads, pool.head_dim):
        raise ValueError("the bounds are of another pool's shape")
    B, shape = start_pos.numel(), block_table.shape
    if len(shape) != 2 or shape[0] != B or cu_new.numel() != B + 1:
        raise ValueError("start_pos and block_table hold one entry (row) per sequence, cu_new one more")
    rc = lib().nk_page_bounds(pool._struct(), bounds.storage.data_ptr(), block_table.data_ptr(), shape[1],
                              start_pos.data_ptr(), cu_new.data_ptr(), B, _ptr(status), _stream(stream))
    _check(rc, "nk_page_bounds")


def page_select_workspace_bytes(B: int, T: int, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                                max_ctx: int) -> int:
    return int(lib().nk_page_select_workspace_bytes(B, T, num_q_heads, num_kv_heads, head_dim, page_size, max_ctx))


def _large(*n):
    raise ValueError(f"sizes and counts must lie between 0 and 2^31 - 1, not {n}")


def page_select(bounds: PageBounds, q, block_table, ctx_lens, page_size: int, max_ctx: int, k: int, sink_pages: int = 1,
                recent_pages: int = 1, workspace=None, out=None, status=None, stream=None):
    """The ``k`` pages of each query token and kv-head whose bounds promise the
    largest scores (nk_page_select): ``q`` bf16 [B][T][Hq][D]; returns int32
    [B][T][Hkv][k], ascending, -1 behind the last."""
    import torch

    _need(torch.bfloat16, q)
    _need(torch.int32, block_table, ctx_lens, out, status)
    _need_scratch(bounds.storage, workspace)
    bounds._check()
    if not (-1 < page_size <= _I32_MAX and -1 < max_ctx <= _I32_MAX and -1 < k <= _I32_MAX and -1 < sink_pages <= _I32_MAX
            and -1 < recent_pages <= _I32_MAX):
        _large(page_size, max_ctx, k, sink_pages, recent_pages)
    B, T, Hq, D = q.shape
    Hkv, shape = bounds.num_kv_heads, block_table.shape
    if D != bounds.head_dim or len(shape) != 2 or shape[0] != B or ctx_lens.numel() != B:
        raise ValueError("q, block_table, ctx_lens and the bounds disagree on the batch or the head dim")
    if out is None:
        out = _empty(stream, block_table, (B, T, Hkv, k), torch.int32)
    elif out.numel() != B * T * Hkv * k:
        raise ValueError("out must be [B][T][kv-heads][k]")
    if workspace is None:
        wbytes = lib().nk_page_select_workspace_bytes(B, T, Hq, Hkv, D, page_size, max_ctx)
        if wbytes > 0:
            workspace = _empty(stream, q, wbytes, torch.uint8)
    else:
        wbytes = workspace.numel() * workspace.element_size()
    rc = lib().nk_page_select(bounds.storage.data_ptr(), bounds.num_pages, page_size, Hkv, D, q.data_ptr(),
                              block_table.data_ptr(), shape[1], ctx_lens.data_ptr(), B, T, Hq, max_ctx, k, sink_pages,
                              recent_pages, _ptr(workspace), wbytes, out.data_ptr(), _ptr(status), _stream(stream))
    _check(rc, "nk_page_select")
    return out


def paged_sparse_attn(pool: KVPool, q, block_table, ctx_lens, pages, sm_scale: float, max_ctx: int, num_ctas: int = 0,
                      workspace=None, out=None, status=None, stream=None):
    """Decode / verify attention over the listed ``pages`` int32 [B][T][Hkv][k]
    of each query token and kv-head (nk_paged_sparse_attn; page_select makes
    such lists); returns out bf16 [B][T][Hq][D]."""
    import torch

    _need(torch.bfloat16, q, out)
    _need(torch.int32, block_table, ctx_lens, pages, status)
    _need_scratch(pool.storage, workspace)
    pool.need("int8")
    if not (-1 < max_ctx <= _I32_MAX and -_I32_MAX <= num_ctas <= _I32_MAX):
        _large(max_ctx, num_ctas)
    B, T, Hq, D = q.shape
    shape, lists, Hkv = block_table.shape, pages.shape, pool.num_kv_heads
    if D != pool.head_dim or len(shape) != 2 or shape[0] != B or ctx_lens.numel() != B:
        raise ValueError("q, block_table, ctx_lens and the pool disagree on the batch or the head dim")
    if len(lists) != 4 or lists[:3] != (B, T, Hkv):
        raise ValueError("pages must be [B][T][kv-heads][pages]")
    if lists[3] > _I32_MAX:
        _large(lists[3])
    if out is None:
        out = _empty(stream, q, q.shape)
    elif out.numel() != q.numel():
        raise ValueError("out must have the shape of q")
    if workspace is None:
        wbytes = max(lib().nk_decode_workspace_bytes(B * T, 1, Hq, Hkv, D, num_ctas), 256)
        workspace = _empty(stream, q, wbytes, torch.uint8)
    else:
        wbytes = workspace.numel() * workspace.element_size()
    rc = lib().nk_paged_sparse_attn(pool._struct(), q.data_ptr(), block_table.data_ptr(), shape[1], ctx_lens.data_ptr(),
                                    pages.data_ptr(), lists[3], B, T, Hq, sm_scale, max_ctx, num_ctas,
                                    workspace.data_ptr(), wbytes, out.data_ptr(), _ptr(status), _stream(stream))
    _check(rc, "nk_paged_sparse_attn")
    return out


def page_weights_workspace_bytes(B: int, T: int, num_q_heads: int, num_kv_heads: int, page_size: int,
                                 max_ctx: int) -> int:
    return int(lib().nk_page_weights_workspace_bytes(B, T, num_q_heads, num_kv_heads, page_size, max_ctx))


def page_weights(pool: KVPool, q, block_table, ctx_lens, sm_scale: float, max_ctx: int, weights, prior=None, seen=None,
                 workspace=None, status=None, stream=None):
    """The attention weight that each page of the batch draws from ``q`` bf16
    [B][T][Hq][D], added to ``prior`` (nk_page_weights): ``weights`` fp32
    [num_pages][Hkv] is written for the batch's pages and returned; pass it as
    ``prior`` too to accumulate in place, with ``seen`` int32 [B] the tokens that
    earlier calls covered."""
    import torch

    _need(torch.bfloat16, q)
    _need(torch.float32, weights, prior)
    _need(torch.int32, block_table, ctx_lens, seen, status)
    _need_scratch(pool.storage, workspace)
    pool.need("int8")
    if not -1 < max_ctx <= _I32_MAX:
        _large(max_ctx)
    B, T, Hq, D = q.shape
    shape, Hkv = block_table.shape, pool.num_kv_heads
    if D != pool.head_dim or len(shape) != 2 or shape[0] != B or ctx_lens.numel() != B:
        raise ValueError("q, block_table, ctx_lens and the pool disagree on the batch or the head dim")
    if seen is not None and seen.numel() != B:
        raise ValueError("seen must hold one count per sequence")
    for t in (weights, prior):
        if t is not None and t.shape != (pool.num_pages, Hkv):
            raise ValueError("weights and prior must be [num_pages][kv-heads]")
    if workspace is None:
        wbytes = lib().nk_page_weights_workspace_bytes(B, T, Hq, Hkv, pool.page_size, max_ctx)
        workspace = _empty(stream, q, max(wbytes, 16), torch.uint8)
    else:
        wbytes = workspace.numel() * workspace.element_size()
    rc = lib().nk_page_weights(pool._struct(), q.data_ptr(), block_table.data_ptr(), shape[1], ctx_lens.data_ptr(), B, T,
                               Hq, sm_scale, max_ctx, _ptr(prior), _ptr(seen), workspace.data_ptr(), wbytes,
                               weights.data_ptr(), _ptr(status), _stream(stream))
    _check(rc, "nk_page_weights")
    return weights


def evict_pages(page_size: int, weights, block_table, ctx_lens, keep_pages: int, new_ctx, freed, num_freed,
                sink_pages: int = 1, recent_pages: int = 1, out=None, status=None, stream=None):
    """Cuts sequences back to the ``keep_pages`` pages that drew the most
    attention (nk_evict_pages): ``weights`` fp32 [num_pages][Hkv], the compacted
    table in ``out`` (default: ``block_table`` itself, in place), ``new_ctx``
    int32 [B], the pages given back in ``freed`` int32 and their count in
    ``num_freed`` int32 [1]. Returns the table."""
    import torch

    if out is None:
        out = block_table
    _need(torch.float32, weights)
    _need(torch.int32, block_table, ctx_lens, new_ctx, freed, num_freed, out, status)
    if not (-1 < page_size <= _I32_MAX and -1 < keep_pages <= _I32_MAX and -1 < sink_pages <= _I32_MAX
            and -1 < recent_pages <= _I32_MAX):
        _large(page_size, keep_pages, sink_pages, recent_pages)
    _one(num_freed, "num_freed")
    B, shape = ctx_lens.numel(), block_table.shape
    if len(shape) != 2 or shape[0] != B or out.shape != shape or new_ctx.numel() != B or weights.dim() != 2:
        raise ValueError("block_table, out, ctx_lens and new_ctx hold one row (entry) per sequence, weights are [num_pages][kv-heads]")
    rc = lib().nk_evict_pages(page_size, weights.shape[0], weights.shape[1], weights.data_ptr(), block_table.data_ptr(),
                              out.data_ptr(), shape[1], ctx_lens.data_ptr(), B, keep_pages, sink_pages, recent_pages,
                              new_ctx.data_ptr(), freed.data_ptr(), min(freed.numel(), _I32_MAX), num_freed.data_ptr(),
                              _ptr(status), _stream(stream))
    _check(rc, "nk_evict_pages")
    return out


def _vocab_stride(t, what: str) -> int:
    """Elements between the rows of [B][rows][vocab], which must all be the same distance apart."""
    if t.is_contiguous():
        return t.shape[2]
    (b, r, v), (s0, s1, s2) = t.shape, t.stride()
    if v > 1 and s2 != 1:
        raise ValueError(f"the entries of a row of {what} must be consecutive")
    row = s1 if r > 1 else (s0 if b > 1 else v)
    if b > 1 and r > 0 and s0 != r * row:
        raise ValueError(f"the rows of {what} must all be the same distance apart")
    return row


def verify_drafts(target, draft, drafts, uniforms, num_drafts=None, ctx_lens=None, next_start=None, tokens=None,
                  accepted=None, status=None, stream=None):
    """Accepts or replaces drafted tokens (nk_verify_drafts): ``target`` fp32
    [B][T][vocab] and ``draft`` [B][T-1][vocab] (None: certain drafts) are
    probabilities, ``drafts`` int32 [B][T-1], ``uniforms`` fp32 [B][T]. Returns
    (tokens int32 [B][T], accepted int32 [B]); with ``ctx_lens`` int32 [B],
    ``next_start`` int32 [B] gets the cache rows that stand."""
    import torch

    shape = target.shape
    if len(shape) != 3 or shape[1] < 1 or (draft is not None and draft.shape != (shape[0], shape[1] - 1, shape[2])):
        raise ValueError("target must be [B][T][vocab] and draft [B][T-1][vocab]")
    B, T, V = shape
    if V > _I32_MAX:
        _large(V)
    here = _here()
    for t in (target, draft):
        if t is not None and not (t.get_device() == here and t.dtype == torch.float32):
            _refuse(t, here, torch.float32)
    _need(torch.float32, uniforms)
    _need(torch.int32, drafts, num_drafts, ctx_lens, next_start, tokens, accepted, status)
    if drafts.numel() != B * (T - 1) or uniforms.numel() != B * T:
        raise ValueError("drafts must be [B][T-1] and uniforms [B][T]")
    for t in (num_drafts, ctx_lens, next_start, accepted):
        if t is not None and t.numel() != B:
            raise ValueError("num_drafts, ctx_lens, next_start and accepted hold one entry per sequence")
    if tokens is None:
        tokens = _empty(stream, drafts, (B, T), torch.int32)
    elif tokens.numel() != B * T:
        raise ValueError("tokens must be [B][T]")
    if accepted is None:
        accepted = _empty(stream, drafts, (B,), torch.int32)
    rc = lib().nk_verify_drafts(target.data_ptr(), _vocab_stride(target, "target"), _ptr(draft),
                                0 if draft is None else _vocab_stride(draft, "draft"), drafts.data_ptr(),
                                _ptr(num_drafts), uniforms.data_ptr(), B, T, V, _ptr(ctx_lens), tokens.data_ptr(),
                                accepted.data_ptr(), _ptr(next_start), _ptr(status), _stream(stream))
    _check(rc, "nk_verify_drafts")
    return tokens, accepted
