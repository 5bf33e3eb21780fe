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
import struct

import torch

from . import _binding as _b

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
# b200attn_paged_cache of the header
_CACHE = struct.Struct("@2P6q6i2P")


def _is_cuda(t):
    return isinstance(t, torch.Tensor) and t.is_cuda


def _check_ints(name, t, shape, device):
    if not (_is_cuda(t) and t.dtype is _I32 and t.shape == shape and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {device}")


def _check_table(t, batch, device):
    """The row stride of a block table."""
    if not (_is_cuda(t) and t.dtype is _I32 and t.dim() == 2 and t.device == device):
        raise ValueError(f"block_table must be a 2-D int32 tensor on {device}")
    (rows, width), (row, col) = t.shape, t.stride()
    if rows != batch or width < 1:
        raise ValueError(f"block_table must have shape [{batch}, pages], got {tuple(t.shape)}")
    if rows == 1:
        row = width
    if (width > 1 and col != 1) or row < width:
        raise ValueError("block_table must have contiguous rows that do not overlap")
    return row


def _check_rows(name, t, heads, d, device):
    """bf16 [tokens, heads, d], each token contiguous, tokens any multiple of 8
    elements apart (a slice of a fused projection's output): their distance."""
    if not (_is_cuda(t) and t.dtype is _BF16 and t.dim() == 3 and t.device == device):
        raise ValueError(f"{name} must be a 3-D bf16 tensor on {device}")
    (_, h, dim), (token, head, one) = t.shape, t.stride()
    if (heads is not None and h != heads) or h < 1 or dim != d:
        raise ValueError(f"{name} must have shape [tokens, {heads or 'heads'}, {d}], got {tuple(t.shape)}")
    if one != 1 or (h > 1 and head != d) or token % 8 != 0:
        raise ValueError(f"{name} must have contiguous heads and a token stride that is a multiple of 8 elements")
    return token


def _strides(name, c, esz):
    """(page, token, head) strides in elements; those of dimensions of one are replaced by what they would be."""
    (P, ps, H, d), (page, token, head, one) = c.shape, c.stride()
    if P == 1:
        page = ps * H * d
    if ps == 1:
        token = H * d
    if H == 1:
        head = d
    if one != 1:
        raise ValueError(f"{name} must have contiguous rows (d fastest)")
    if page <= 0 or token <= 0 or head <= 0 or (page | token | head) * esz & 15:
        raise ValueError(f"{name}'s strides must be positive multiples of 16 bytes")
    return page, token, head


def _cache(k_cache, v_cache, k_scale, v_scale):
    """Checks the cache tensors: (description for the library, Hkv, d_qk, d_v)."""
    if not (_is_cuda(k_cache) and _is_cuda(v_cache)):
        raise ValueError("k_cache and v_cache must be CUDA tensors")
    if k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be 4-D [pages, page_size, H, d]")
    dev, dtype = k_cache.device, k_cache.dtype
    (P, ps, H, d_qk), d_v = k_cache.shape, v_cache.shape[3]
    if v_cache.device != dev:
        raise ValueError("k_cache and v_cache must be on one device")
    if v_cache.shape != (P, ps, H, d_v) or v_cache.dtype is not dtype:
        raise ValueError("k_cache and v_cache must agree in pages, page_size, heads and dtype")
    if P < 1 or ps < 1 or H < 1:
        raise ValueError("the cache must hold at least one page, row and head")
    if dtype is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales are for e4m3 caches")
        esz, code, ks, vs = 2, _b.BF16, 0, 0
    elif _b._is_fp8(k_cache):
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is None:
                raise ValueError(f"{name} is required for an e4m3 cache")
            if not (_is_cuda(s) and s.dtype is _F32 and s.shape == (H,) and s.device == dev and s.is_contiguous()):
                raise ValueError(f"{name} must be contiguous fp32 [{H}] on {dev}")
        esz, code, ks, vs = 1, _b.FP8_E4M3, k_scale.data_ptr(), v_scale.data_ptr()
    else:
        raise ValueError("the cache must be bf16 or e4m3")
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), *_strides("k_cache", k_cache, esz),
                       *_strides("v_cache", v_cache, esz), P, ps, H, d_qk, d_v, code, ks, vs), H, d_qk, d_v


_HERE = contextlib.nullcontext()


def _on(device):
    """The tensors' device as the current one."""
    if device.type != "cuda" or device.index == torch._C._cuda_getDevice():
        return _HERE
    return torch.cuda.device(device)


def _stream(stream, device):
    """The stream to launch on: the current one of the tensors' device by default."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return _b._stream_handle(stream)


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
    if not _is_cuda(context_lens) or context_lens.dim() != 1 or context_lens.shape[0] < 1:
        raise ValueError("context_lens must be an int32 [batch] CUDA tensor")
    B, dev = context_lens.shape[0], context_lens.device
    _check_ints("context_lens", context_lens, (B,), dev)
    _check_ints("new_lens", new_lens, (B,), dev)
    row = _check_table(block_table, B, dev)
    total, page_size = int(total), int(page_size)
    if total < 0 or page_size < 1:
        raise ValueError("total must not be negative and page_size at least 1")
    free, count, head, head_out = None, 0, None, None
    if free_pages is not None:
        if not _is_cuda(free_pages) or free_pages.dim() != 1:
            raise ValueError("free_pages must be an int32 [pages] CUDA tensor")
        count = free_pages.shape[0]
        _check_ints("free_pages", free_pages, (count,), dev)
        _check_ints("free_head", free_head, (1,), dev)
        if free_head_out is not None:
            _check_ints("free_head_out", free_head_out, (1,), dev)
        head = free_head.data_ptr()
        free = free_pages.data_ptr() or head  # an empty list needs an address; none of it is read
    elif free_head is not None or free_head_out is not None:
        raise ValueError("free_head goes with free_pages")
    out = torch.empty(2 * B + 2 + 2 * total, dtype=_I32, device=dev)
    cu, kv, pos, slots, new_head = out.split_with_sizes((B + 1, B, total, total, 1))
    at = out.data_ptr()
    if free_pages is not None:
        if free_head_out is None:
            free_head_out = new_head
        head_out = free_head_out.data_ptr()
    with _on(dev):
        _done(lib.b200attn_paged_slots(
            block_table.data_ptr(), row, block_table.shape[1], context_lens.data_ptr(), new_lens.data_ptr(), B, total,
            page_size, free, count, head, head_out, at, at + 4 * (B + 1), at + 4 * (2 * B + 1),
            at + 4 * (2 * B + 1 + total), _stream(stream, dev)), "b200attn_paged_slots")
    return (cu, kv, pos, slots) if free_pages is None else (cu, kv, pos, slots, free_head_out)


def paged_append_kv(k, v, k_cache, v_cache, slots, *, k_scale=None, v_scale=None, stream=None):
    """Writes the rows of k [total, Hkv, d_qk] and v [total, Hkv, d_v] (bf16; slices of a fused projection's output
    are taken as they are) to the cache rows ``slots`` (int32 [total]; negative: the row is skipped), as bf16 or as
    e4m3(x / scale) with one fp32 scale per head, via b200attn_paged_append. Returns (k_cache, v_cache)."""
    lib = _b.load_library()
    cache, H, d_qk, d_v = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    k_row = _check_rows("k", k, H, d_qk, dev)
    v_row = _check_rows("v", v, H, d_v, dev)
    total = k.shape[0]
    if v.shape[0] != total:
        raise ValueError("k and v must have the same number of tokens")
    _check_ints("slots", slots, (total,), dev)
    with _on(dev):
        _done(lib.b200attn_paged_append(k.data_ptr(), v.data_ptr(), k_row, v_row, total, cache, slots.data_ptr(),
                                        _stream(stream, dev)), "b200attn_paged_append")
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
    cache, Hkv, d_qk, d_v = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    q_row = _check_rows("q", q, None, d_qk, dev)
    total, Hq, _ = q.shape
    if Hq % Hkv != 0:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    if not _is_cuda(kv_lens) or kv_lens.dim() != 1 or kv_lens.shape[0] < 1:
        raise ValueError("kv_lens must be an int32 [batch] CUDA tensor")
    B = kv_lens.shape[0]
    _check_ints("kv_lens", kv_lens, (B,), dev)
    _check_ints("cu_seqlens", cu_seqlens, (B + 1,), dev)
    row = _check_table(block_table, B, dev)
    max_q = total if max_seqlen_q is None else int(max_seqlen_q)
    if max_q < 1 and total > 0:
        raise ValueError("max_seqlen_q must be at least 1")
    if out is None:
        out = torch.empty((total, Hq, d_v), dtype=_BF16, device=dev)
    else:
        _b._check_buffer("out", out, (total, Hq, d_v), (_BF16,), dev)
    lse = torch.empty((Hq, total), dtype=_F32, device=dev) if return_lse else None
    if total == 0:
        return (out, lse) if return_lse else out
    max_q = min(max_q, total)
    if workspace is None:
        size = lib.b200attn_paged_fwd_workspace_bytes(total, max_q, Hq, Hkv)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    else:
        if not _is_cuda(workspace) or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {dev}")
        size = workspace.numel() * workspace.element_size()
    with _on(dev):
        _done(lib.b200attn_paged_fwd(
            q.data_ptr(), q_row, cache, block_table.data_ptr(), row, block_table.shape[1], cu_seqlens.data_ptr(),
            kv_lens.data_ptr(), B, total, max_q, Hq, 1 if causal else 0, float(softmax_scale) if softmax_scale else 0.0,
            out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(), size, _stream(stream, dev)),
              "b200attn_paged_fwd")
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
