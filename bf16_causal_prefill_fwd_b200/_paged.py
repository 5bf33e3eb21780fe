"""Serving from a paged key/value cache (b200attn_paged_* of include/b200attn.h):
argument checks and marshalling, as in _binding.py.

A cache is two tensors, k_cache [pages, page_size, Hkv, d_qk] and v_cache
[pages, page_size, Hkv, d_v], bf16 or e4m3 (torch.float8_e4m3fn or uint8 codes)
with one fp32 scale per key/value head. They may be views (a [pages, Hkv,
page_size, d] buffer permuted, K and V halves of one buffer): rows of d elements
are contiguous, the other strides are multiples of 16 bytes.

Lengths, tables and slots are int32 CUDA tensors read on the device only: no call
here copies from the device or waits for it, so each can be captured into a CUDA
graph and replayed on new contents. Work goes to the current stream of the
tensors' device, whichever device is current.

A decoding step makes these calls once per layer, with kernels of a few
microseconds, so the checks read each tensor's properties once and build error
texts only when they fail.
"""
from __future__ import annotations

import struct

import torch

from . import _binding as _b

_BF16, _F32, _I32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
_CACHE = struct.Struct("@2P6q6i2P")  # b200attn_paged_cache of the header
_device_of = torch.Tensor.get_device  # -1: not on a GPU
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _need(ok, name, what, t):
    if not ok:
        got = f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name} must be {what}, got {got}")


def _ints(name, t, shape, dev):
    """Address of a contiguous int32 tensor of `shape` on GPU `dev`."""
    try:
        if t.dtype is _I32 and t.shape == shape and _device_of(t) == dev and t.is_contiguous():
            return t.data_ptr()
    except (AttributeError, TypeError):
        pass
    _need(False, name, f"a contiguous int32 tensor of shape {tuple(shape)} on cuda:{dev}", t)


def _batch(name, t):
    """(batch, device) of an int32 [batch] tensor."""
    try:
        dev = _device_of(t)
        if dev >= 0 and t.dtype is _I32 and t.dim() == 1 and t.shape[0] > 0:
            return t.shape[0], dev
    except (AttributeError, TypeError):
        pass
    _need(False, name, "a contiguous int32 [batch] CUDA tensor", t)


def _table(t, batch, dev):
    """(row stride, width) of a block table."""
    try:
        if t.dtype is _I32 and _device_of(t) == dev:
            (rows, width), (row, col) = t.shape, t.stride()
            if rows == 1:
                row = width
            if rows == batch and width > 0 and (col == 1 or width == 1) and row >= width:
                return row, width
    except (AttributeError, TypeError, ValueError):
        pass
    _need(False, "block_table", f"int32 [{batch}, pages] on cuda:{dev} with contiguous rows that do not overlap", t)


def _rows(name, t, d, dev):
    """(tokens, heads, distance of tokens) of bf16 [tokens, heads, d], each token contiguous, tokens any multiple of 8
    elements apart (a slice of a fused projection's output)."""
    try:
        if t.dtype is _BF16 and _device_of(t) == dev:
            (n, h, dim), (token, head, one) = t.shape, t.stride()
            if dim == d and h > 0 and one == 1 and (head == d or h == 1) and token % 8 == 0:
                return n, h, token
    except (AttributeError, TypeError, ValueError):
        pass
    _need(False, name, f"bf16 [tokens, heads, {d}] on cuda:{dev} with contiguous heads and a token stride that is a "
                       "multiple of 8 elements", t)


def _cache(k, v, k_scale, v_scale):
    """Checks the cache tensors: (description for the library, device, Hkv, d_qk, d_v)."""
    try:
        dev, dtype = _device_of(k), k.dtype
        (P, ps, H, d_qk), (page, token, head, one) = k.shape, k.stride()
        (vP, vps, vH, d_v), (vpage, vtoken, vhead, vone) = v.shape, v.stride()
        fine = dev >= 0 and _device_of(v) == dev and v.dtype is dtype and one == 1 and vone == 1
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        raise ValueError("k_cache and v_cache must be 4-D [pages, page_size, H, d] CUDA tensors of one dtype and device, "
                         "d fastest")
    if vP != P or vps != ps or vH != H or P < 1 or ps < 1 or H < 1:
        raise ValueError("k_cache and v_cache must agree in pages, page_size and heads, at least one of each")
    if dtype is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales are for e4m3 caches")
        esz, code, ks, vs = 2, _b.BF16, 0, 0
    elif dtype is _E4M3 or dtype is _U8:
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is None:
                raise ValueError(f"{name} is required for an e4m3 cache")
            if not (isinstance(s, torch.Tensor) and s.dtype is _F32 and s.shape == (H,) and _device_of(s) == dev
                    and s.is_contiguous()):
                _need(False, name, f"contiguous fp32 [{H}] on cuda:{dev}", s)
        esz, code, ks, vs = 1, _b.FP8_E4M3, k_scale.data_ptr(), v_scale.data_ptr()
    else:
        raise ValueError("the cache must be bf16 or e4m3")
    # a dimension of one may come with any stride: what it would be
    if P == 1:
        page, vpage = ps * H * d_qk, ps * H * d_v
    if ps == 1:
        token, vtoken = H * d_qk, H * d_v
    if H == 1:
        head, vhead = d_qk, d_v
    if ((page | token | head | vpage | vtoken | vhead) * esz & 15
            or min(page, token, head, vpage, vtoken, vhead) <= 0):
        raise ValueError("k_cache's and v_cache's strides must be positive multiples of 16 bytes")
    return (_CACHE.pack(k.data_ptr(), v.data_ptr(), page, token, head, vpage, vtoken, vhead, P, ps, H, d_qk, d_v, code,
                        ks, vs), dev, H, d_qk, d_v)


def _run(name, fn, dev, stream, *args):
    """Calls the library with the tensors' device current, on its current stream or `stream`."""
    if dev == _current_device():
        rc = fn(*args, _raw_stream(dev) if stream is None else _b._stream_handle(stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev) if stream is None else _b._stream_handle(stream))
    if rc != 0:
        raise _b.B200AttnError(rc, name)


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
    lib = _b._lib or _b.load_library()
    B, dev = _batch("context_lens", context_lens)
    ctx = _ints("context_lens", context_lens, (B,), dev)
    new = _ints("new_lens", new_lens, (B,), dev)
    row, width = _table(block_table, B, dev)
    if total < 0 or page_size < 1:
        raise ValueError("total must not be negative and page_size at least 1")
    free, count, head, head_out = None, 0, None, None
    if free_pages is not None:
        count = free_pages.numel() if isinstance(free_pages, torch.Tensor) else 0
        free = _ints("free_pages", free_pages, (count,), dev)
        head = _ints("free_head", free_head, (1,), dev)
        if count == 0:
            free = head  # an empty list needs an address; none of it is read
        if free_head_out is not None:
            head_out = _ints("free_head_out", free_head_out, (1,), dev)
    elif free_head is not None or free_head_out is not None:
        raise ValueError("free_head goes with free_pages")
    # one allocation: int32 cu_seqlens, kv_lens, positions, slots, head
    out = context_lens.new_empty(2 * B + 2 + 2 * total)
    cu, kv, pos, slots, new_head = out.split_with_sizes((B + 1, B, total, total, 1))
    at = out.data_ptr()
    if free is not None and free_head_out is None:
        free_head_out, head_out = new_head, at + 4 * (2 * B + 1 + 2 * total)
    _run("b200attn_paged_slots", lib.b200attn_paged_slots, dev, stream, block_table.data_ptr(), row, width, ctx, new, B,
         total, page_size, free, count, head, head_out, at, at + 4 * (B + 1), at + 4 * (2 * B + 1),
         at + 4 * (2 * B + 1 + total))
    return (cu, kv, pos, slots) if free is None else (cu, kv, pos, slots, free_head_out)


def paged_append_kv(k, v, k_cache, v_cache, slots, *, k_scale=None, v_scale=None, stream=None):
    """Writes the rows of k [total, Hkv, d_qk] and v [total, Hkv, d_v] (bf16; slices of a fused projection's output
    are taken as they are) to the cache rows ``slots`` (int32 [total]; negative: the row is skipped), as bf16 or as
    e4m3(x / scale) with one fp32 scale per head, via b200attn_paged_append. Returns (k_cache, v_cache)."""
    lib = _b._lib or _b.load_library()
    cache, dev, H, d_qk, d_v = _cache(k_cache, v_cache, k_scale, v_scale)
    total, kh, k_row = _rows("k", k, d_qk, dev)
    vn, vh, v_row = _rows("v", v, d_v, dev)
    if kh != H or vh != H or vn != total:
        raise ValueError(f"k and v must have the cache's {H} heads and the same number of tokens")
    at = _ints("slots", slots, (total,), dev)
    _run("b200attn_paged_append", lib.b200attn_paged_append, dev, stream, k.data_ptr(), v.data_ptr(), k_row, v_row, total,
         cache, at)
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
    lib = _b._lib or _b.load_library()
    cache, dev, Hkv, d_qk, d_v = _cache(k_cache, v_cache, k_scale, v_scale)
    total, Hq, q_row = _rows("q", q, d_qk, dev)
    if Hq % Hkv != 0:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    B, _ = _batch("kv_lens", kv_lens)
    kv = _ints("kv_lens", kv_lens, (B,), dev)
    cu = _ints("cu_seqlens", cu_seqlens, (B + 1,), dev)
    row, width = _table(block_table, B, dev)
    max_q = total if max_seqlen_q is None else min(int(max_seqlen_q), total)
    if max_q < 1 and total > 0:
        raise ValueError("max_seqlen_q must be at least 1")
    if out is None:
        out = q.new_empty((total, Hq, d_v))
    else:
        _b._check_buffer("out", out, (total, Hq, d_v), (_BF16,), q.device)
    lse = torch.empty((Hq, total), dtype=_F32, device=q.device) if return_lse else None
    if total == 0:
        return (out, lse) if return_lse else out
    if workspace is None:
        size = lib.b200attn_paged_fwd_workspace_bytes(total, max_q, Hq, Hkv)
        workspace = kv_lens.new_empty((size + 3) // 4)
    else:
        if not isinstance(workspace, torch.Tensor) or _device_of(workspace) != dev or not workspace.is_contiguous():
            _need(False, "workspace", f"contiguous on cuda:{dev}", workspace)
        size = workspace.numel() * workspace.element_size()
    _run("b200attn_paged_fwd", lib.b200attn_paged_fwd, dev, stream, q.data_ptr(), q_row, cache, block_table.data_ptr(), row,
         width, cu, kv, B, total, max_q, Hq, 1 if causal else 0, float(softmax_scale) if softmax_scale else 0.0,
         out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(), size)
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
