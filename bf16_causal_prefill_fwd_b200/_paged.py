"""Serving from a paged key/value cache (b200attn_paged_* of include/b200attn.h).

A cache is two tensors, k_cache [pages, page_size, Hkv, d_qk] and v_cache
[pages, page_size, Hkv, d_v], bf16 or e4m3 (torch.float8_e4m3fn or uint8 codes)
with one positive fp32 scale per key/value head. They may be views (a [pages, Hkv,
page_size, d] buffer permuted, K and V halves of one buffer): rows of d elements
are contiguous, the other strides are multiples of 16 bytes. page_size is a multiple
of 16 (any for paged_slots alone).

Lengths, tables and slots are int32 CUDA tensors read on the device only: no call
here copies from the device or waits for it, so each can be captured into a CUDA
graph and replayed on new contents (a workspace or output given to a captured call
has to live as long as the graph). Work goes to the current stream of the tensors'
device, whichever device is current, or to ``stream`` (a torch.cuda.Stream or a raw
handle). What a call allocates then belongs to that stream, as under
torch.cuda.stream(stream), and results are recorded on the caller's current stream as
well; the inputs have to be ready there, and to live until the work is done.

The checks and the marshalling are compiled (csrc/paged_binding.cpp): a decoding
step makes these calls once per layer around kernels of a few microseconds.
Arguments that do not fit raise ValueError, a status of the library B200AttnError.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

from . import _binding as _b

BINDING_PATH = os.path.join(os.path.dirname(_b.LIB_PATH), "_paged_binding.so")
_native = None


def _bind(module) -> None:
    """Gives the compiled part the addresses of the library's functions."""
    lib = _b.load_library()
    fns = (lib.b200attn_paged_slots, lib.b200attn_paged_append, lib.b200attn_paged_fwd,
           lib.b200attn_paged_fwd_workspace_bytes)
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in fns), False)


def _load():
    global _native
    if _native is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is missing; build it with `python -m bf16_causal_prefill_fwd_b200.build`")
        from .build import binding_built_for, binding_stamp

        if binding_stamp() not in (None, binding_built_for()):
            raise RuntimeError(f"{BINDING_PATH} was built for {binding_stamp()}, this is {binding_built_for()}; "
                               "build it with `python -m bf16_causal_prefill_fwd_b200.build`")
        loader = importlib.machinery.ExtensionFileLoader("_paged_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_paged_binding", loader))
        loader.exec_module(module)
        _bind(module)
        _native = module
    return _native


def _stream(stream):
    return None if stream is None else _b._stream_handle(stream)


def paged_slots(block_table, context_lens, new_lens, total: int, page_size: int, *, free_pages=None, free_head=None,
                free_head_out=None, stream=None):
    """A step's bookkeeping via b200attn_paged_slots: from context_lens and new_lens (int32 [B]: tokens cached and
    new) to (cu_seqlens [B+1], kv_lens [B], positions [total], slots [total]), all int32.

    ``total`` is the number of token rows the step is run with; rows behind the last new token get slot -1. With
    ``free_pages`` (int32 page numbers) the pages the new tokens need are taken from entry free_head[0] on and
    written into block_table, and a fifth result holds the new head (``free_head_out``, which may be free_head
    itself, or a new tensor). Results that are not given are parts of one allocation, each contiguous, which lives
    as long as any of them. A step that does not fit is empty, and check() says why: -1 for lengths that do not
    fit, -6 for too few free pages.
    """
    r = (_native or _load()).slots(block_table, context_lens, new_lens, total, page_size, free_pages, free_head,
                                   free_head_out, _stream(stream))
    if r.__class__ is int:
        raise _b.B200AttnError(r, "b200attn_paged_slots")
    return r


def paged_append_kv(k, v, k_cache, v_cache, slots, *, k_scale=None, v_scale=None, stream=None):
    """Writes the rows of k [total, Hkv, d_qk] and v [total, Hkv, d_v] (bf16; slices of a fused projection's output
    are taken as they are) to the cache rows ``slots`` (int32 [total]; negative: the row is skipped), as bf16 or as
    e4m3(x / scale) with one fp32 scale per head, via b200attn_paged_append. Returns (k_cache, v_cache)."""
    rc = (_native or _load()).append(k, v, k_cache, v_cache, slots, k_scale, v_scale, _stream(stream))
    if rc != 0:
        raise _b.B200AttnError(rc, "b200attn_paged_append")
    return k_cache, v_cache


def attn_paged_workspace_bytes(total: int, max_seqlen_q: int, Hq: int, Hkv: int) -> int:
    """Bytes of a workspace for attn_paged_fwd with `total` rows of q; enough for fewer rows and tokens as well."""
    return int(_b.load_library().b200attn_paged_fwd_workspace_bytes(total, max_seqlen_q, Hq, Hkv))


def attn_paged_fwd(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, *, max_seqlen_q: int | None = None,
                   causal: bool = True, softmax_scale: float | None = None, k_scale=None, v_scale=None, out=None,
                   return_lse: bool = False, workspace=None, stream=None):
    """Attention of new tokens over their requests' pages via b200attn_paged_fwd.

    q [total, Hq, d_qk] bf16 holds each request's new tokens, request b's at cu_seqlens[b]:cu_seqlens[b+1];
    kv_lens [B] counts its keys, the new tokens' own included (append them first). With ``causal`` new token i of nq
    sees the keys j <= kv_len - nq + i. ``max_seqlen_q`` bounds the new tokens of any request (default: total); with
    at most 16 / (Hq / Hkv) of them the decoding kernel runs. Returns bf16 [total, Hq, d_v] (and fp32 lse
    [Hq, total]); rows of no request are left unwritten. ``out``, if given,
    is contiguous and 32-byte aligned.
    """
    r = (_native or _load()).fwd(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_seqlen_q, causal, softmax_scale,
                                 k_scale, v_scale, out, return_lse, workspace, _stream(stream))
    if r.__class__ is int:
        raise _b.B200AttnError(r, "b200attn_paged_fwd")
    return r


def attn_paged_func(q, k, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens, slots, softmax_scale: float | None = None,
                    causal: bool = True, *, max_seqlen_q: int | None = None, k_scale=None, v_scale=None, out=None,
                    return_lse: bool = False, workspace=None, stream=None):
    """One layer's attention of a serving step: paged_append_kv of the new K and V rows, then attn_paged_fwd of the
    new queries over the pages (cu_seqlens, kv_lens and slots as paged_slots gives them; out and workspace as
    attn_paged_fwd takes them)."""
    paged_append_kv(k, v, k_cache, v_cache, slots, k_scale=k_scale, v_scale=v_scale, stream=stream)
    return attn_paged_fwd(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_seqlen_q=max_seqlen_q,
                          causal=causal, softmax_scale=softmax_scale, k_scale=k_scale, v_scale=v_scale, out=out,
                          return_lse=return_lse, workspace=workspace, stream=stream)
