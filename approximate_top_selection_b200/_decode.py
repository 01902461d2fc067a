"""Binding of the decoding step's operators: the paged key-value cache,
attention over it, and beam search (include/topk_b200.h).

As in _binding.py: argument checks and marshalling only, all work runs in the
CUDA library.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import (TOPK_CACHE_BF16, TOPK_CACHE_E4M3, TopkCache, _check, _cuda, _OnDevice, _stream_handle,
                       load_library)

_E4M3 = torch.float8_e4m3fn


def _cuda_strided(t: torch.Tensor, name: str, dtype, dims: int) -> None:
    """As _cuda, for a tensor that needs contiguous elements in its last dimension only."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != dims:
        raise ValueError("%s must have %d dimensions" % (name, dims))
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)


def _same_device(first: torch.Tensor, **others) -> None:
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError("%s is on %s, not on %s" % (name, t.device, first.device))


def _cache(data: torch.Tensor, scale, name: str) -> TopkCache:
    """The C description of a cache tensor [pages, kv_heads, page_size, d]."""
    if isinstance(data, torch.Tensor) and data.dtype == _E4M3:
        kind = TOPK_CACHE_E4M3
        _cuda_strided(data, name, _E4M3, 4)
        if scale is None:
            raise ValueError("%s is e4m3 and needs its scale" % name)
        if not isinstance(scale, torch.Tensor) or not scale.is_cuda or scale.dtype != torch.float32:
            raise TypeError("the scale of %s must be a float32 CUDA tensor" % name)
        if tuple(scale.shape) != tuple(data.shape[:3]):
            raise ValueError("the scale of %s must be [pages, kv_heads, page_size]" % name)
        _same_device(data, scale=scale)
    else:
        kind = TOPK_CACHE_BF16
        _cuda_strided(data, name, torch.bfloat16, 4)
        if scale is not None:
            raise ValueError("%s is bfloat16 and takes no scale" % name)
    pages, heads, page, d = data.shape
    c = TopkCache(data.data_ptr(), scale.data_ptr() if scale is not None else None, pages, heads, page, d, kind,
                  *data.stride()[:3], *(scale.stride() if scale is not None else (0, 0, 0)))
    return c


def _two_caches(k_cache, v_cache, k_scale, v_scale):
    kc, vc = _cache(k_cache, k_scale, "k_cache"), _cache(v_cache, v_scale, "v_cache")
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must have the same shape and dtype")
    _same_device(k_cache, v_cache=v_cache)
    return kc, vc


def _table(block_table, seq_lens, batch):
    _cuda_strided(block_table, "block_table", torch.int32, 2)
    _cuda(seq_lens, "seq_lens", torch.int32)
    if block_table.shape[0] != batch or seq_lens.numel() != batch:
        raise ValueError("block_table must be [batch, width] and seq_lens [batch]")
    if block_table.shape[1] < 1:
        raise ValueError("block_table needs a column at least")


# Workspace of paged_attention and topk_beam: one per (device, stream) for
# calls that run at once; its first part is zero before and after every call,
# the rest is scratch.  A call under stream capture gets one of its own from
# the graph's memory instead, so that graphs (which may be replayed on other
# streams, side by side) share none.
_ws_cache: dict = {}


def _workspace(nbytes: int, device: torch.device, stream: int):
    if nbytes == 0:
        return None
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, stream)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def _pointer(t):
    return t.data_ptr() if t is not None else None


def paged_attention_workspace_bytes(batch: int, heads: int, lists: int, d: int) -> int:
    """Workspace bytes of a paged_attention call on the current device (lists = 0 without positions)."""
    return int(load_library().paged_attention_workspace_bytes(batch, heads, lists, d))


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, *, scale: float | None = None, k_scale=None, v_scale=None,
                    positions=None, return_lse: bool = False, out=None, out_lse=None,
                    workspace: torch.Tensor | None = None, stream=None):
    """Attention of one new token per sequence over a paged key-value cache.

    q: [batch, heads, d] bfloat16.  k_cache, v_cache: [pages, kv_heads,
    page_size, d] bfloat16, or float8_e4m3fn with k_scale, v_scale [pages,
    kv_heads, page_size] float32; heads is a multiple of kv_heads.  block_table:
    [batch, width] int32 page numbers; seq_lens: [batch] int32.  positions:
    None for all tokens, or [batch, lists, c] int32 token positions (as
    score_topk and score_rerank return them; negative = empty), list l serving
    heads l * heads / lists and on.  scale: 1 / sqrt(d) unless given.
    Returns out [batch, heads, d] bfloat16, or (out, lse [batch, heads]
    float32).  A head with nothing to attend to gives zeros and -inf.
    """
    lib = load_library()
    _cuda_strided(q, "q", torch.bfloat16, 3)
    batch, heads, d = q.shape
    if heads > 1 and q.stride(1) != d:
        raise ValueError("the heads of q must be contiguous")
    kc, vc = _two_caches(k_cache, v_cache, k_scale, v_scale)
    if k_cache.shape[3] != d:
        raise ValueError("q and the caches disagree on d")
    if heads % k_cache.shape[1]:
        raise ValueError("heads must be a multiple of kv_heads")
    _table(block_table, seq_lens, batch)
    lists = c = 0
    if positions is not None:
        _cuda(positions, "positions", torch.int32)
        if positions.dim() != 3 or positions.shape[0] != batch:
            raise ValueError("positions must be [batch, lists, c]")
        lists, c = positions.shape[1:]
        if lists < 1 or c < 1 or lists % k_cache.shape[1] or heads % lists:
            raise ValueError("positions needs c >= 1 and lists a multiple of kv_heads that divides heads")
    _same_device(q, k_cache=k_cache, block_table=block_table, seq_lens=seq_lens, positions=positions, out=out,
                 out_lse=out_lse, workspace=workspace)
    with _OnDevice(q.device, stream) as on:
        sh = _stream_handle(stream, on.index)
        if out is None:
            out = torch.empty(batch, heads, d, dtype=torch.bfloat16, device=q.device)
        _cuda(out, "out", torch.bfloat16)
        if out_lse is None and return_lse:
            out_lse = torch.empty(batch, heads, dtype=torch.float32, device=q.device)
        if out_lse is not None:
            _cuda(out_lse, "out_lse", torch.float32)
        if out.numel() != q.numel() or (out_lse is not None and out_lse.numel() != batch * heads):
            raise ValueError("out must hold batch*heads*d elements and out_lse batch*heads")
        ws = workspace
        if ws is None:
            ws = _workspace(paged_attention_workspace_bytes(batch, heads, lists, d), q.device, sh)
        st = lib.paged_attention(
            q.data_ptr(), q.stride(0), batch, heads, ctypes.byref(kc), ctypes.byref(vc), block_table.data_ptr(),
            block_table.stride(0), block_table.shape[1], seq_lens.data_ptr(), _pointer(positions), lists, c,
            d ** -0.5 if scale is None else float(scale), out.data_ptr(), _pointer(out_lse), _pointer(ws),
            ws.numel() if ws is not None else 0, sh)
    _check(st, "paged_attention")
    return (out, out_lse) if return_lse else out


def cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
                *, k_scale=None, v_scale=None, stream=None) -> None:
    """Write new tokens' keys and values into a paged cache, quantising them if it is e4m3.

    k, v: [tokens, kv_heads, d] bfloat16 (strides over tokens and heads are
    free: slices of a projection's output need no copy).  slots: [tokens] int64,
    page * page_size + offset; negative = not written.  The slots of one call
    must be distinct.  Caches and scales as in paged_attention; an e4m3 row
    gets the smallest power-of-two scale that holds it.
    """
    lib = load_library()
    _cuda_strided(k, "k", torch.bfloat16, 3)
    _cuda_strided(v, "v", torch.bfloat16, 3)
    kc, vc = _two_caches(k_cache, v_cache, k_scale, v_scale)
    if k.shape != v.shape or tuple(k.shape[1:]) != (k_cache.shape[1], k_cache.shape[3]):
        raise ValueError("k and v must be [tokens, kv_heads, d]")
    _cuda(slots, "slots", torch.int64)
    if slots.dim() != 1 or slots.numel() != k.shape[0]:
        raise ValueError("slots must be [tokens]")
    _same_device(k, v=v, k_cache=k_cache, slots=slots)
    with _OnDevice(k.device, stream) as on:
        sh = _stream_handle(stream, on.index)
        st = lib.cache_write(k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                             k.shape[0], ctypes.byref(kc), ctypes.byref(vc), slots.data_ptr(), sh)
    _check(st, "cache_write")


def cache_read(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, n: int, *, scale=None,
               out=None, stream=None) -> torch.Tensor:
    """The first n tokens of every sequence as contiguous rows [batch, kv_heads, n, d] bfloat16.

    Rows behind a sequence's end are zeros.  `out.view(-1, n, d)` is the key
    matrix per row that score_topk and score_rerank take.
    """
    lib = load_library()
    c = _cache(cache, scale, "cache")
    batch = seq_lens.numel() if isinstance(seq_lens, torch.Tensor) else 0
    _table(block_table, seq_lens, batch)
    _same_device(cache, block_table=block_table, seq_lens=seq_lens, out=out)
    shape = (batch, cache.shape[1], int(n), cache.shape[3])
    with _OnDevice(cache.device, stream) as on:
        sh = _stream_handle(stream, on.index)
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
        _cuda(out, "out", torch.bfloat16)
        if tuple(out.shape) != shape:
            raise ValueError("out must be [batch, kv_heads, n, d]")
        st = lib.cache_read(ctypes.byref(c), block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
                            seq_lens.data_ptr(), batch, int(n), out.data_ptr(), sh)
    _check(st, "cache_read")
    return out


def topk_beam_workspace_bytes(batch: int, beams: int, n: int, k: int) -> int:
    """Workspace bytes of a topk_beam call on the current device."""
    return int(load_library().topk_beam_workspace_bytes(batch, beams, n, k))


def topk_beam(logits: torch.Tensor, beam_scores: torch.Tensor, k: int, *, out_scores=None, out_parent=None,
              out_token=None, workspace: torch.Tensor | None = None, stream=None):
    """One step of beam search: the k best continuations of each sentence's beams.

    logits: [batch, beams, n] float32 or bfloat16; beam_scores: [batch, beams]
    float32 (-inf = the beam has ended).  A continuation of beam i by token t is
    worth beam_scores[i] + log_softmax(logits[i])[t].  Returns (scores float32,
    parents int32, tokens int32), each [batch, k], best first, padded with
    -inf, -1, -1.
    """
    lib = load_library()
    bf16 = isinstance(logits, torch.Tensor) and logits.dtype == torch.bfloat16
    _cuda(logits, "logits", torch.bfloat16 if bf16 else torch.float32)
    _cuda(beam_scores, "beam_scores", torch.float32)
    if logits.dim() != 3 or tuple(beam_scores.shape) != tuple(logits.shape[:2]):
        raise ValueError("logits must be [batch, beams, n] and beam_scores [batch, beams]")
    _same_device(logits, beam_scores=beam_scores, out_scores=out_scores, out_parent=out_parent, out_token=out_token,
                 workspace=workspace)
    batch, beams, n = logits.shape
    with _OnDevice(logits.device, stream) as on:
        sh = _stream_handle(stream, on.index)
        outs = []
        for t, name, dtype in ((out_scores, "out_scores", torch.float32), (out_parent, "out_parent", torch.int32),
                               (out_token, "out_token", torch.int32)):
            if t is None:
                t = torch.empty(batch, k, dtype=dtype, device=logits.device)
            _cuda(t, name, dtype)
            if t.numel() != batch * k:
                raise ValueError("outputs must hold batch*k elements")
            outs.append(t)
        ws = workspace
        if ws is None:
            ws = _workspace(topk_beam_workspace_bytes(batch, beams, n, k), logits.device, sh)
        fn = lib.topk_beam_bf16 if bf16 else lib.topk_beam
        st = fn(logits.data_ptr(), beam_scores.data_ptr(), batch, beams, n, k, *(t.data_ptr() for t in outs),
                _pointer(ws), ws.numel() if ws is not None else 0, sh)
    _check(st, "topk_beam")
    return tuple(outs)


def beam_reorder(states, parents: torch.Tensor, *, out=None, stream=None):
    """Per-beam states in the order topk_beam chose.

    states: a contiguous tensor [batch, beams, ...] of any dtype, or a list or
    tuple of up to 256 of them; parents: [batch, k] int32.  Returns the same
    with [batch, k, ...]: row (b, j) is row (b, parents[b, j]), zeros where
    that is -1.  `out` (of the same form) must not overlap the states.
    """
    lib = load_library()
    one = isinstance(states, torch.Tensor)
    src = [states] if one else list(states)
    _cuda(parents, "parents", torch.int32)
    if not src or parents.dim() != 2:
        raise ValueError("states needs a tensor at least and parents must be [batch, k]")
    for t in src:
        _cuda(t, "states", t.dtype if isinstance(t, torch.Tensor) else None)
        if t.dim() < 2 or tuple(t.shape[:2]) != tuple(src[0].shape[:2]) or t.shape[0] != parents.shape[0]:
            raise ValueError("every state must be [batch, beams, ...]")
        if t.numel() == 0:
            raise ValueError("states must not be empty")
        _same_device(parents, states=t)
    batch, k = parents.shape
    beams = src[0].shape[1]
    with _OnDevice(parents.device, stream) as on:
        sh = _stream_handle(stream, on.index)
        if out is None:
            dst = [torch.empty((batch, k) + tuple(t.shape[2:]), dtype=t.dtype, device=t.device) for t in src]
        else:
            dst = [out] if isinstance(out, torch.Tensor) else list(out)
            if len(dst) != len(src):
                raise ValueError("out needs one tensor per state")
            for t, o in zip(src, dst):
                _cuda(o, "out", t.dtype)
                _same_device(t, out=o)
                if tuple(o.shape) != (batch, k) + tuple(t.shape[2:]):
                    raise ValueError("out must be [batch, k, ...]")
        m = len(src)
        pointers = ctypes.c_void_p * m
        size = (ctypes.c_int64 * m)(*(t.numel() // (batch * beams) * t.element_size() for t in src))
        st = lib.beam_reorder(pointers(*(t.data_ptr() for t in src)), pointers(*(t.data_ptr() for t in dst)), size, m,
                              batch, beams, k, parents.data_ptr(), sh)
    _check(st, "beam_reorder")
    return dst[0] if one else dst
