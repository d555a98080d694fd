"""Exact attention (FlashAttention-2 formulation) for GB300 / sm_103a.

The computation lives in ``libfa.so`` (hand-written CUDA: TMA, tcgen05 MMA
with tensor-memory accumulators, warp-specialised softmax), reached through
its C ABI (``include/fa.h``).  This package is the thin Python side: the
ctypes binding (``_lib``), convenience wrappers that allocate outputs with
PyTorch, the seeded input generators (``inputs``) and the build script.

PyTorch is used for device memory and streams only.  There is no CPU or
eager fallback: if the library is missing the calls raise.
"""
from __future__ import annotations

import math

from . import _lib

__all__ = ["attention_fwd", "attention_bwd", "attention_fwd_varlen", "attention_bwd_varlen",
           "hadamard_quant_fp8", "attention_fwd_fp8", "paged_tables", "paged_append", "attention_fwd_paged",
           "attention_fwd_paged_prefix", "attention_fwd_paged_tree", "paged_fork", "paged_copy", "paged_compact", "paged_free"]


def _default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def attention_fwd(q, k, v, causal: bool = False, scale: float | None = None, stream=None,
                  window: int | None = None):
    """Returns (O, LSE).  q [B,Hq,N,d], k/v [B,Hkv,N,d]: contiguous CUDA
    bf16/fp16 tensors; LSE is fp32 [B,Hq,N] (natural log).  ``window`` (with
    causal=True) limits row r to keys r - window + 1 .. r."""
    import torch
    B, Hq, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    sc = _default_scale(d) if scale is None else scale
    if window is None:
        _lib.fa_fwd(q, k, v, o, lse, causal, sc, stream)
    else:
        if not causal:
            raise ValueError("a sliding window is defined on top of the causal mask")
        _lib.fa_fwd_local(q, k, v, o, lse, window, sc, stream)
    return o, lse


def attention_bwd(q, k, v, o, lse, dO, causal: bool = False, scale: float | None = None,
                  workspace=None, stream=None, deterministic: bool = False, window: int | None = None):
    """Returns (dQ, dK, dV) from the forward's O and LSE and the incoming dO.

    ``deterministic=True`` forms dQ in a second pass over Q tiles instead of
    by atomic addition (bit-identical results from run to run)."""
    import torch
    B, Hq, N, d = q.shape
    if workspace is None:
        size_fn = _lib.fa_bwd_two_pass_workspace_bytes if deterministic else _lib.fa_bwd_workspace_bytes
        workspace = torch.empty(size_fn(B, Hq, N, d), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    sc = _default_scale(d) if scale is None else scale
    if window is not None:
        if not causal:
            raise ValueError("a sliding window is defined on top of the causal mask")
        _lib.fa_bwd_local(q, k, v, o, lse, dO, dq, dk, dv, window, sc, deterministic, workspace, stream)
    else:
        fn = _lib.fa_bwd_two_pass if deterministic else _lib.fa_bwd
        fn(q, k, v, o, lse, dO, dq, dk, dv, causal, sc, workspace, stream)
    return dq, dk, dv


def attention_fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int | None = None, causal: bool = False,
                         scale: float | None = None, window: int | None = None, stream=None):
    """Packed batch: sequence b is rows cu_seqlens[b] .. cu_seqlens[b+1]-1 of
    q [total,Hq,d] and k/v [total,Hkv,d] and attends only within itself.
    ``cu_seqlens`` is an int32 tensor [B+1] on the device.  Returns
    (O [total,Hq,d], LSE [Hq,total] fp32).  ``max_seqlen`` defaults to the
    longest sequence (read back from the device once)."""
    import torch
    total, Hq, d = q.shape
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    if window is not None and not causal:
        raise ValueError("a sliding window is defined on top of the causal mask")
    o = torch.empty_like(q)
    lse = torch.empty((Hq, total), dtype=torch.float32, device=q.device)
    sc = _default_scale(d) if scale is None else scale
    _lib.fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen, causal, sc, window or 0, stream)
    return o, lse


def attention_bwd_varlen(q, k, v, o, lse, dO, cu_seqlens, max_seqlen: int | None = None, causal: bool = False,
                         scale: float | None = None, window: int | None = None, deterministic: bool = False,
                         workspace=None, stream=None):
    """Gradients (dQ [total,Hq,d], dK, dV [total,Hkv,d]) of a packed batch
    from the forward's O and LSE and the incoming dO; arguments as
    ``attention_fwd_varlen``.  ``deterministic=True`` forms dQ in a second
    pass instead of by atomic addition."""
    import torch
    total, Hq, d = q.shape
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    if window is not None and not causal:
        raise ValueError("a sliding window is defined on top of the causal mask")
    if workspace is None:
        workspace = torch.empty(_lib.fa_bwd_varlen_workspace_bytes(total, Hq, d, deterministic),
                                dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    sc = _default_scale(d) if scale is None else scale
    _lib.fa_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens, max_seqlen, causal, sc, deterministic,
                       workspace, window or 0, stream)
    return dq, dk, dv


def hadamard_quant_fp8(x, signs=None, stream=None):
    """Random-sign Hadamard rotation (if ``signs`` is given) and per-tensor
    e4m3 quantisation of a bf16 tensor [..., d].  Returns (x8, descale)."""
    import torch
    d = x.shape[-1]
    x8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    descale = torch.empty(1, dtype=torch.float32, device=x.device)
    ws = torch.empty(_lib.fa_hadamard_quant_workspace_bytes(x.numel() // d, d), dtype=torch.uint8,
                     device=x.device)
    _lib.fa_hadamard_quant_fp8(x, signs, x8, descale, ws, stream)
    return x8, descale


def attention_fwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, causal: bool = False,
                      scale: float | None = None, stream=None):
    """FP8 forward: bf16 O and fp32 LSE from e4m3 Q, K, V and their descales."""
    import torch
    B, Hq, N, d = q8.shape
    o = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q8.device)
    _lib.fa_fwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, o, lse, causal,
                    _default_scale(d) if scale is None else scale, stream)
    return o, lse


def _on(stream):
    """Makes `stream` the current one: outputs are allocated on the stream
    that writes them."""
    import torch
    if isinstance(stream, int):
        # torch takes the handle 0, the default stream's, for a request for a new one
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def paged_tables(cached_lens, new_lens, block_table, free_pages, page_size: int, num_pages: int, total: int,
                 free_start=None, stream=None):
    """Hands pages to each request's new tokens and maps the tokens to slots.

    All tensors are int32 on the device: ``cached_lens`` and ``new_lens`` [B],
    ``block_table`` [B,max_pages] (its new cells are filled in place),
    ``free_pages`` the pool's unused pages, of which those from position
    ``free_start`` (one element; default 0) on are handed out.  ``total`` is
    the number of rows to map, at least the sum of ``new_lens``.  Returns
    (seq_lens [B], cu_seqlens [B+1], slots [total], counts [2]): lengths with
    the new tokens, row offsets, a slot per row (-1 for rows behind the last
    request and for requests the pool had no pages for), and the next
    ``free_start`` with the number of pages lacking."""
    if stream is not None:
        with _on(stream):
            return paged_tables(cached_lens, new_lens, block_table, free_pages, page_size, num_pages, total, free_start)
    if total > 0x7FFFFFFF:
        raise ValueError(f"total: {total} does not fit 32 bits")
    B, empty = block_table.shape[0], block_table.new_empty
    seq_lens, cu_seqlens, slots, counts = empty(B), empty(B + 1), empty(total), empty(2)
    _lib.fa_paged_tables(cached_lens, new_lens, free_pages, free_start, block_table, seq_lens, cu_seqlens, slots,
                         counts, page_size, num_pages)
    return seq_lens, cu_seqlens, slots, counts


def paged_append(k, v, slots, k_cache, v_cache, stream=None):
    """Writes k, v [total,Hkv,d] into the slots of k_cache, v_cache
    [pages,Hkv,page_size,d] in place; a negative slot skips its row, and no
    slot may occur twice."""
    _lib.fa_paged_append(k, v, slots, k_cache, v_cache, stream)


def paged_fork(src, dst, seq_lens, block_table, free_pages, shares, page_size: int, free_start=None, stream=None):
    """Lets requests branch: row dst[f] of ``block_table`` [B,max_pages]
    continues where row src[f] stands, on the same pages but for a half-full
    last one, in whose place it gets a page of the pool.

    All tensors are int32 on the device.  ``seq_lens`` [B], ``block_table``
    and ``shares`` [pages] (how many requests hold a page beside the first)
    are updated in place; ``free_pages`` and ``free_start`` are those of
    ``paged_tables``.  No row may occur twice in ``dst``, or in both.  Returns
    (copies [3,F], counts [2]): source page, new page and rows to copy for
    each fork, to be given to ``paged_copy`` for every layer's cache (-1, -1,
    0 where nothing is to be copied), and the next ``free_start`` with the
    number of pages lacking.  A fork that the pool had no page for gets
    length 0.  Pages that row dst[f] held before are not given back: end its
    request by ``paged_free`` first."""
    if stream is not None:
        with _on(stream):
            return paged_fork(src, dst, seq_lens, block_table, free_pages, shares, page_size, free_start)
    copies, counts = src.new_empty((3, src.numel())), src.new_empty(2)
    _lib.fa_paged_fork(src, dst, seq_lens, block_table, free_pages, free_start, shares, copies, counts, page_size)
    return copies, counts


def paged_copy(src, dst, k_cache, v_cache, rows=None, stream=None):
    """Copies the first rows[i] tokens (default: all) of page src[i] to page
    dst[i] of k_cache, v_cache [pages,Hkv,page_size,d], in place.  Negative
    page numbers skip the pair; no page may occur twice in ``dst``, or in
    both."""
    _lib.fa_paged_copy(src, dst, rows, k_cache, v_cache, stream)


def paged_compact(keep, keep_lens, base_lens, block_table, k_cache, v_cache, stream=None):
    """Moves the kept ones of each request's last tokens together, in place:
    token base_lens[b] + keep[b][i] becomes token base_lens[b] + i, for
    i < keep_lens[b].  ``keep`` [B,max_keep] is strictly increasing within a
    request: the accepted path of a tree of drafted tokens, or what is left of
    a long context.  Tokens may only move to pages that no other request holds:
    on one that ``paged_fork`` shared, the other holders' tokens would be
    overwritten, and nothing reports it.  (A branch's shared pages lie before
    the place where it branched, its drafted tokens behind.)  int32 tensors;
    the request has base_lens + keep_lens tokens then (``paged_free`` takes the
    pages behind them back)."""
    _lib.fa_paged_compact(keep, keep_lens, base_lens, block_table, k_cache, v_cache, stream)


def paged_free(old_lens, new_lens, block_table, free_pages, free_start, page_size: int, num_pages: int, shares=None,
               stream=None):
    """Takes the pages behind new_lens [B] back from requests that had
    old_lens [B] tokens (a request that ends keeps 0).  The lengths are the
    caller's: they have to become new_lens before the next call that reads
    them, or it takes pages that are in the pool for the request's.

    All tensors are int32 on the device.  A page that ``shares`` [num_pages]
    says further requests hold loses holders, and is freed only with its last
    one; without ``shares`` no page is shared.  Freed pages are put into
    ``free_pages`` in front of position ``free_start`` [1] (where the pool's
    entries that were handed out before lie), in order of request and page.
    Returns counts [2]: the next ``free_start``, and how many pages found no
    room there."""
    if stream is not None:
        with _on(stream):
            return paged_free(old_lens, new_lens, block_table, free_pages, free_start, page_size, num_pages, shares)
    counts = block_table.new_empty(2)
    _lib.fa_paged_free(old_lens, new_lens, block_table, free_pages, free_start, shares, counts, page_size, num_pages)
    return counts


def _most_rows(cu_seqlens) -> int:
    """Rows of the request that has the most, read back from the device."""
    most = 1 if cu_seqlens is None else int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    if most == 0:
        raise ValueError("no request has a row")
    return most


def _paged_buffers(q, k_cache, block_table, cu_seqlens, max_new, window, prefix_len, workspace):
    """(O, LSE, workspace, max_new) of a paged forward call."""
    import torch
    if window is not None and window < 1:
        raise ValueError("window must be at least 1")
    total, Hq, d = q.shape
    B, max_pages = block_table.shape
    if max_new is None:
        max_new = _most_rows(cu_seqlens)
    o = torch.empty_like(q)
    lse = torch.empty((Hq, total), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = _lib.fa_fwd_paged_workspace_bytes(B, total, max_new, Hq, k_cache.shape[1], d, max_pages, k_cache.shape[2],
                                              prefix_len)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    return o, lse, workspace, max_new


def attention_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, max_new: int | None = None,
                        scale: float | None = None, window: int | None = None, workspace=None, stream=None):
    """Attention of new tokens to a paged cache that holds their keys and
    values.  q [total,Hq,d]: request b's rows are cu_seqlens[b] ..
    cu_seqlens[b+1]-1, or row b alone without ``cu_seqlens``; the last of them
    sees all seq_lens[b] keys, each row before it one less (``window`` leaves
    a row its last ``window`` ones).  ``max_new`` bounds a request's rows
    (default: the longest, read back from the device once).  ``workspace``: a
    uint8 tensor of at least ``_lib.fa_fwd_paged_workspace_bytes(B, total,
    max_new, Hq, Hkv, d, max_pages, page_size, prefix_len)`` bytes, of which
    calls that may run at once need one each (default: one is allocated).
    Returns (O [total,Hq,d], LSE [Hq,total] fp32); rows of no request stay
    unwritten."""
    if stream is not None:
        with _on(stream):
            return attention_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, max_new, scale, window,
                                       workspace)
    o, lse, workspace, max_new = _paged_buffers(q, k_cache, block_table, cu_seqlens, max_new, window, 0, workspace)
    _lib.fa_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, o, lse, max_new,
                      _default_scale(q.shape[-1]) if scale is None else scale, workspace, window or 0)
    return o, lse


def attention_fwd_paged_prefix(q, k_cache, v_cache, prefix_pages, prefix_len: int, block_table, seq_lens,
                               cu_seqlens=None, max_new: int | None = None, scale: float | None = None,
                               window: int | None = None, workspace=None, stream=None):
    """``attention_fwd_paged`` for requests that all begin with the same
    ``prefix_len`` tokens, stored once on ``prefix_pages`` (int32, on the
    device): where that saves work it is read once for the whole batch.
    ``block_table`` and ``seq_lens`` describe each request's own keys behind
    it."""
    if stream is not None:
        with _on(stream):
            return attention_fwd_paged_prefix(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, seq_lens,
                                              cu_seqlens, max_new, scale, window, workspace)
    o, lse, workspace, max_new = _paged_buffers(q, k_cache, block_table, cu_seqlens, max_new, window, prefix_len,
                                                workspace)
    _lib.fa_fwd_paged_prefix(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, seq_lens, cu_seqlens, o,
                             lse, max_new, _default_scale(q.shape[-1]) if scale is None else scale, workspace,
                             window or 0)
    return o, lse


def attention_fwd_paged_tree(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, parents, max_new: int | None = None,
                             scale: float | None = None, window: int | None = None, workspace=None, stream=None):
    """``attention_fwd_paged`` for trees of drafted tokens, whose keys are the
    last ones of each request.  ``parents`` (int32 [total], on the device):
    the row of its request, counted from 0, that a row's token follows, below
    its own, or -1 where it follows the context.  A row sees the context, its
    path up to there and itself (``window``: the last ``window`` tokens of
    these).  At most 1024 rows a request; paths of hundreds of tokens take many
    times as long as the same rows in ``attention_fwd_paged``.  ``workspace``: as there, of
    ``_lib.fa_fwd_paged_tree_workspace_bytes(B, total, max_new, Hq, Hkv, d,
    max_pages, page_size)`` bytes."""
    if stream is not None:
        with _on(stream):
            return attention_fwd_paged_tree(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, parents, max_new,
                                            scale, window, workspace)
    if window is not None and window < 1:
        raise ValueError("window must be at least 1")
    if max_new is None:
        max_new = _most_rows(cu_seqlens)
    return _lib.paged_tree_forward(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, parents, max_new,
                                   _default_scale(q.shape[-1]) if scale is None else scale, window or 0, workspace)
