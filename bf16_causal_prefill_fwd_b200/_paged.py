"""Serving from a paged key/value cache (b200attn_paged_* of include/b200attn.h):
argument checks and marshalling, as in _binding.py.

A cache is two tensors, k_cache [pages, page_size, Hkv, d_qk] and v_cache
[pages, page_size, Hkv, d_v], bf16 or e4m3 (torch.float8_e4m3fn or uint8 codes)
with one fp32 scale per key/value head. They may be views (a [pages, Hkv,
page_size, d] buffer permuted, K and V halves of one buffer): rows of d elements
are contiguous, the other strides are multiples of 16 bytes.

Lengths, tables and slots are int32 CUDA tensors read on the device only: no call
here copies from the device or waits for it, so each can be captured into a CUDA
graph and replayed on new contents.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _binding as _b

_MAX_GROUP = 128


def _check_cuda(name, t, dtype, dim):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D {dtype} tensor")


def _check_ints(name, t, shape, device):
    _check_cuda(name, t, torch.int32, len(shape))
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_table(t, batch, device):
    _check_cuda("block_table", t, torch.int32, 2)
    if t.device != device:
        raise ValueError(f"block_table must be on {device}")
    if t.shape[0] != batch or t.shape[1] < 1:
        raise ValueError(f"block_table must have shape [{batch}, pages], got {tuple(t.shape)}")
    if (t.shape[1] > 1 and t.stride(1) != 1) or (batch > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("block_table must have contiguous rows that do not overlap")


def _check_rows(name, t, heads, d, device):
    """bf16 [tokens, heads, d], each token contiguous, tokens any multiple of 8
    elements apart (a slice of a fused projection's output)."""
    _check_cuda(name, t, torch.bfloat16, 3)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if (heads is not None and t.shape[1] != heads) or t.shape[2] != d:
        raise ValueError(f"{name} must have shape [tokens, {heads or 'heads'}, {d}], got {tuple(t.shape)}")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d) or t.stride(0) % 8 != 0:
        raise ValueError(f"{name} must have contiguous heads and a token stride that is a multiple of 8 elements")


def _strides(name, c):
    """(page, token, head) strides in elements; those of dimensions of one are replaced by what they would be."""
    esz = c.element_size()
    P, ps, H, d = c.shape
    if c.stride(3) != 1:
        raise ValueError(f"{name} must have contiguous rows (d fastest)")
    out = []
    for size, stride, usual in ((P, c.stride(0), ps * H * d), (ps, c.stride(1), H * d), (H, c.stride(2), d)):
        if size == 1:
            stride = usual
        if stride <= 0 or stride * esz % 16 != 0:
            raise ValueError(f"{name}'s strides must be positive multiples of 16 bytes")
        out.append(stride)
    return out


def _cache(k_cache, v_cache, k_scale, v_scale):
    """Checks the cache tensors and describes them to the library."""
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(c, torch.Tensor) or not c.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if c.dim() != 4:
            raise ValueError(f"{name} must be 4-D [pages, page_size, H, d]")
    if k_cache.device != v_cache.device:
        raise ValueError("k_cache and v_cache must be on one device")
    if k_cache.shape[:3] != v_cache.shape[:3] or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must agree in pages, page_size, heads and dtype")
    fp8 = _b._is_fp8(k_cache)
    if not fp8 and k_cache.dtype != torch.bfloat16:
        raise ValueError("the cache must be bf16 or e4m3")
    P, ps, H, d_qk = k_cache.shape
    if min(P, ps, H) < 1:
        raise ValueError("the cache must hold at least one page, row and head")
    if fp8:
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is None:
                raise ValueError(f"{name} is required for an e4m3 cache")
            _check_cuda(name, s, torch.float32, 1)
            if s.device != k_cache.device or s.shape[0] != H or not s.is_contiguous():
                raise ValueError(f"{name} must be contiguous fp32 [{H}] on {k_cache.device}")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales are for e4m3 caches")
    return _b.PagedCache(k_cache.data_ptr(), v_cache.data_ptr(), *_strides("k_cache", k_cache),
                         *_strides("v_cache", v_cache), P, ps, H, d_qk, v_cache.shape[3], _b.FP8_E4M3 if fp8 else _b.BF16,
                         _b._ptr(k_scale) if fp8 else None, _b._ptr(v_scale) if fp8 else None)


def _on(device):
    """The tensors' device as the current one."""
    if device.type != "cuda" or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _done(rc, what):
    if rc != 0:
        raise _b.B200AttnError(rc, what)


def paged_slots(block_table, context_lens, new_lens, total: int, page_size: int, *, free_pages=None, free_head=None,
                free_head_out=None, stream=None):
    """A step's bookkeeping via b200attn_paged_slots: from context_lens and new_lens (int32 [B]: tokens cached and
    new) to (cu_seqlens [B+1], kv_lens [B], positions [total], slots [total]), all int32.

    ``total`` is the number of token rows the step is run with; rows behind the last new token get slot -1. With
    ``free_pages`` (int32 page numbers) the pages the new tokens need are taken from entry free_head[0] on and
    written into block_table, and a fifth result holds the new head (``free_head_out``, which may be free_head
    itself, or a new tensor). A step that does not fit is empty, and check() says why: -1 for lengths that do not
    fit, -6 for too few free pages.
    """
    lib = _b.load_library()
    if not isinstance(context_lens, torch.Tensor) or context_lens.dim() != 1 or context_lens.shape[0] < 1:
        raise ValueError("context_lens must be an int32 [batch] CUDA tensor")
    B, dev = context_lens.shape[0], context_lens.device
    _check_ints("context_lens", context_lens, (B,), dev)
    _check_ints("new_lens", new_lens, (B,), dev)
    _check_table(block_table, B, dev)
    total, page_size = int(total), int(page_size)
    if total < 0 or page_size < 1:
        raise ValueError("total must not be negative and page_size at least 1")
    if free_pages is None:
        if free_head is not None or free_head_out is not None:
            raise ValueError("free_head goes with free_pages")
    else:
        if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
            raise ValueError("free_pages must be an int32 [pages] CUDA tensor")
        _check_ints("free_pages", free_pages, (free_pages.shape[0],), dev)
        _check_ints("free_head", free_head, (1,), dev)
        if free_head_out is None:
            free_head_out = torch.empty(1, dtype=torch.int32, device=dev)
        else:
            _check_ints("free_head_out", free_head_out, (1,), dev)
    out = torch.empty(2 * B + 1 + 2 * total, dtype=torch.int32, device=dev)
    cu, kv, pos, slots = out.split((B + 1, B, total, total))
    if free_pages is not None and free_pages.shape[0] == 0:
        free_pages = torch.zeros(1, dtype=torch.int32, device=dev)  # an address; none of it is free
        count = 0
    else:
        count = 0 if free_pages is None else free_pages.shape[0]
    with _on(dev):
        _done(lib.b200attn_paged_slots(
            _b._ptr(block_table), block_table.stride(0) if B > 1 else block_table.shape[1], block_table.shape[1],
            _b._ptr(context_lens), _b._ptr(new_lens), B, total, page_size, _b._ptr(free_pages), count,
            _b._ptr(free_head), _b._ptr(free_head_out), _b._ptr(cu), _b._ptr(kv), _b._ptr(pos), _b._ptr(slots),
            _b._stream_handle(stream)), "b200attn_paged_slots")
    return (cu, kv, pos, slots) if free_pages is None else (cu, kv, pos, slots, free_head_out)


def paged_append_kv(k, v, k_cache, v_cache, slots, *, k_scale=None, v_scale=None, stream=None):
    """Writes the rows of k [total, Hkv, d_qk] and v [total, Hkv, d_v] (bf16; slices of a fused projection's output
    are taken as they are) to the cache rows ``slots`` (int32 [total]; negative: the row is skipped), as bf16 or as
    e4m3(x / scale) with one fp32 scale per head, via b200attn_paged_append. Returns (k_cache, v_cache)."""
    lib = _b.load_library()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    _check_rows("k", k, c.Hkv, c.d_qk, dev)
    _check_rows("v", v, c.Hkv, c.d_v, dev)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have the same number of tokens")
    _check_ints("slots", slots, (k.shape[0],), dev)
    with _on(dev):
        _done(lib.b200attn_paged_append(_b._ptr(k), _b._ptr(v), k.stride(0), v.stride(0), k.shape[0], ctypes.addressof(c),
                                        _b._ptr(slots), _b._stream_handle(stream)), "b200attn_paged_append")
    return k_cache, v_cache


def attn_paged_workspace_bytes(total: int, max_seqlen_q: int, Hq: int, Hkv: int) -> int:
    return int(_b.load_library().b200attn_paged_fwd_workspace_bytes(total, max_seqlen_q, Hq, Hkv))


def attn_paged_fwd(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, *, max_seqlen_q: int | None = None,
                   causal: bool = True, softmax_scale: float | None = None, k_scale=None, v_scale=None, out=None,
                   return_lse: bool = False, workspace=None, stream=None):
    """Attention of new tokens over their requests' pages via b200attn_paged_fwd.

    q [total, Hq, d_qk] bf16 holds each request's new tokens, request b's at cu_seqlens[b]:cu_seqlens[b+1];
    kv_lens [B] counts its keys, the new tokens' own included (append them first). With ``causal`` new token i of nq
    sees the keys j <= kv_len - nq + i. ``max_seqlen_q`` bounds the new tokens of any request (default: total); with
    at most 16 / (Hq / Hkv) of them the decoding kernel runs. Returns bf16 [total, Hq, d_v] (and fp32 lse
    [Hq, total]); rows of no request are left unwritten.
    """
    lib = _b.load_library()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    _check_rows("q", q, None, c.d_qk, dev)
    total, Hq, _ = q.shape
    if Hq % c.Hkv != 0:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    if not isinstance(kv_lens, torch.Tensor) or kv_lens.dim() != 1 or kv_lens.shape[0] < 1:
        raise ValueError("kv_lens must be an int32 [batch] CUDA tensor")
    B = kv_lens.shape[0]
    _check_ints("kv_lens", kv_lens, (B,), dev)
    _check_ints("cu_seqlens", cu_seqlens, (B + 1,), dev)
    _check_table(block_table, B, dev)
    max_q = total if max_seqlen_q is None else int(max_seqlen_q)
    if max_q < 1 and total > 0:
        raise ValueError("max_seqlen_q must be at least 1")
    if out is None:
        out = torch.empty((total, Hq, c.d_v), dtype=torch.bfloat16, device=dev)
    else:
        _b._check_buffer("out", out, (total, Hq, c.d_v), (torch.bfloat16,), dev)
    lse = torch.empty((Hq, total), dtype=torch.float32, device=dev) if return_lse else None
    if total == 0:
        return (out, lse) if return_lse else out
    max_q = min(max_q, total)
    if workspace is None:
        workspace = torch.empty(max(16, attn_paged_workspace_bytes(total, max_q, Hq, c.Hkv)), dtype=torch.uint8,
                                device=dev)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    with _on(dev):
        _done(lib.b200attn_paged_fwd(
            _b._ptr(q), q.stride(0), ctypes.addressof(c), _b._ptr(block_table),
            block_table.stride(0) if B > 1 else block_table.shape[1], block_table.shape[1], _b._ptr(cu_seqlens),
            _b._ptr(kv_lens), B, total, max_q, Hq, 1 if causal else 0, float(softmax_scale) if softmax_scale else 0.0,
            _b._ptr(out), _b._ptr(lse), _b._ptr(workspace), workspace.numel() * workspace.element_size(),
            _b._stream_handle(stream)), "b200attn_paged_fwd")
    return (out, lse) if return_lse else out


def attn_paged_func(q, k, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens, slots, softmax_scale: float | None = None,
                    causal: bool = True, *, max_seqlen_q: int | None = None, k_scale=None, v_scale=None,
                    return_lse: bool = False, stream=None):
    """One layer's attention of a serving step: paged_append_kv of the new K and V rows, then attn_paged_fwd of the
    new queries over the pages (cu_seqlens, kv_lens and slots as paged_slots gives them)."""
    paged_append_kv(k, v, k_cache, v_cache, slots, k_scale=k_scale, v_scale=v_scale, stream=stream)
    return attn_paged_fwd(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_seqlen_q=max_seqlen_q,
                          causal=causal, softmax_scale=softmax_scale, k_scale=k_scale, v_scale=v_scale,
                          return_lse=return_lse, stream=stream)
