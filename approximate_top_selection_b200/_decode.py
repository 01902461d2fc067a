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

_E4M3, _BF16, _F32, _I32, _I64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32, torch.int64

# A step of a few microseconds on the GPU leaves the host as little time.  So a
# call with nothing given but its inputs goes to the extension module
# _decode_calls, which makes it if everything is as usual; otherwise, and where
# that finds something unusual, the call is checked and made here (get_device is
# -1 on the CPU).
_calls = None


def _usual():
    """The extension module, bound to the CUDA library."""
    global _calls
    if _calls is None:
        lib = load_library()
        try:
            from . import _decode_calls as calls
        except ImportError as e:
            raise ImportError("_decode_calls.so is missing or does not fit this torch: build it with "
                              "`python -m approximate_top_selection_b200.build`") from e
        calls.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.paged_attention, lib.paged_attention_workspace_bytes, lib.cache_write, lib.cache_read, lib.topk_beam,
            lib.topk_beam_bf16, lib.topk_beam_workspace_bytes, lib.beam_reorder)))
        _calls = calls
    return _calls


def _made(result, where: str):
    """The outputs of a call that _decode_calls made, or the error it met."""
    if type(result) is int:
        _check(result, where)
    return result


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


def _int32(**sizes) -> None:
    """Sizes that the C interface takes as int: ctypes would cut off what does not fit."""
    for name, n in sizes.items():
        if not -2 ** 31 <= n < 2 ** 31:
            raise ValueError("%s = %d does not fit 32 bits" % (name, n))


def _check_cache(data: torch.Tensor, scale, name: str) -> None:
    if isinstance(data, torch.Tensor) and data.dtype == _E4M3:
        _cuda_strided(data, name, _E4M3, 4)
        if scale is None:
            raise ValueError("%s is e4m3 and needs its scale" % name)
        if not isinstance(scale, torch.Tensor) or not scale.is_cuda or scale.dtype != _F32:
            raise TypeError("the scale of %s must be a float32 CUDA tensor" % name)
        if tuple(scale.shape) != tuple(data.shape[:3]):
            raise ValueError("the scale of %s must be [pages, kv_heads, page_size]" % name)
        _same_device(data, scale=scale)
    else:
        _cuda_strided(data, name, _BF16, 4)
        if scale is not None:
            raise ValueError("%s is bfloat16 and takes no scale" % name)


def _cache(data: torch.Tensor, scale, name: str, dev: int):
    """The C description of a cache tensor [pages, kv_heads, page_size, d] on
    device `dev`, and its shape."""
    try:
        shape, strides, dtype = data.shape, data.stride(), data.dtype
        good = data.get_device() == dev and len(shape) == 4 and strides[3] == 1
        if dtype is _E4M3:
            good = good and scale.get_device() == dev and scale.dtype is _F32 and scale.shape == shape[:3]
        else:
            good = good and dtype is _BF16 and scale is None
    except (AttributeError, TypeError):
        good = False
    if not good:
        _check_cache(data, scale, name)
        if data.get_device() != dev:
            raise ValueError("%s is on %s, not on cuda:%d" % (name, data.device, dev))
    _int32(kv_heads=shape[1], page_size=shape[2], d=shape[3])
    if scale is None:
        return TopkCache(data.data_ptr(), None, *shape, TOPK_CACHE_BF16, *strides[:3], 0, 0, 0), shape
    return TopkCache(data.data_ptr(), scale.data_ptr(), *shape, TOPK_CACHE_E4M3, *strides[:3], *scale.stride()), shape


def _two_caches(k_cache, v_cache, k_scale, v_scale, dev):
    (kc, ks), (vc, vs) = _cache(k_cache, k_scale, "k_cache", dev), _cache(v_cache, v_scale, "v_cache", dev)
    if ks != vs or kc.type != vc.type:
        raise ValueError("k_cache and v_cache must have the same shape and dtype")
    return kc, vc, ks


def _table(block_table, seq_lens, batch, dev):
    """Checks the block table and the lengths; returns (stride, width) of the table."""
    try:
        (rows, width), (stride, inner) = block_table.shape, block_table.stride()
        if (block_table.get_device() == dev and block_table.dtype is _I32 and inner == 1 and rows == batch and width > 0
                and seq_lens.get_device() == dev and seq_lens.dtype is _I32 and seq_lens.shape == (batch,)
                and width < 2 ** 31 and (batch == 1 or seq_lens.stride() == (1,))):
            return stride, width
    except (AttributeError, TypeError, ValueError):
        pass
    _cuda_strided(block_table, "block_table", _I32, 2)
    _cuda(seq_lens, "seq_lens", _I32)
    if block_table.shape[0] != batch or seq_lens.numel() != batch:
        raise ValueError("block_table must be [batch, width] and seq_lens [batch]")
    if block_table.shape[1] < 1:
        raise ValueError("block_table needs a column at least")
    _int32(width=block_table.shape[1])
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        if t.get_device() != dev:
            raise ValueError("%s is on %s, not on cuda:%d" % (name, t.device, dev))
    return block_table.stride(0), block_table.shape[1]


def _device_of(t, name: str) -> int:
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise TypeError("%s must be a CUDA tensor" % name)
    return dev


def _on(dev: int, stream, body, *args):
    """body(*args, stream handle) with `dev` current and, if given, `stream` as torch's current stream."""
    if stream is None and torch._C._cuda_getDevice() == dev:
        return body(*args, torch._C._cuda_getCurrentRawStream(dev))
    with _OnDevice(torch.device("cuda", dev), stream) as on:
        return body(*args, _stream_handle(stream, on.index))


def _out(t, shape, dtype, name: str, dev: int):
    """A given output, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=_devices[dev])
    _cuda(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError("%s is on %s, not on cuda:%d" % (name, t.device, dev))
    n = 1
    for x in shape:
        n *= x
    if t.numel() != n:
        raise ValueError("%s must hold %d elements" % (name, n))
    return t


_devices = [torch.device("cuda", i) for i in range(64)]


# Workspace of paged_attention: one per (device, stream) for calls that run at
# once; its first part is zero before and after every call, the rest is scratch.
# Host threads may share a stream, and then its workspace: a call is one launch,
# so theirs follow one another.  (topk_beam is two launches, between which
# another thread's may come: every call takes scratch of its own.)  A call
# under stream capture gets one of its own from the graph's memory instead, so
# that graphs (which may be replayed on other streams, side by side) share none.
_ws_cache: dict = {}
_WS_ZERO = 16384  # TOPK_DECODE_TICKET_BYTES


def _workspace(nbytes: int, dev: int, stream: int):
    if torch._C._cuda_isCurrentStreamCapturing():
        ws = torch.empty(max(nbytes, _WS_ZERO), dtype=torch.uint8, device=_devices[dev])
        ws[:_WS_ZERO].zero_()
        return ws
    ws = _ws_cache.get((dev, stream))
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=_devices[dev])
        _ws_cache[(dev, stream)] = ws
    return ws


_ws_bytes: dict = {}


def _workspace_bytes(query, *sizes) -> int:
    """A workspace query for the current device, asked once per sizes."""
    key = (torch._C._cuda_getDevice(), query, sizes)
    n = _ws_bytes.get(key)
    if n is None:
        if len(_ws_bytes) > 4096:
            _ws_bytes.clear()
        n = _ws_bytes[key] = query(*sizes)
    return n


def _given_workspace(t, first: torch.Tensor) -> None:
    """A workspace handed in: its bytes have to be there, so no view of fewer."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _same_device(first, workspace=t)


def _bytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


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
    score_topk and score_rerank return them; negative = empty, at or behind the
    sequence's end = left out), list l serving heads l * heads / lists and on.
    scale: 1 / sqrt(d) unless given.
    The table's width stands for the longest length: a slice of the columns that
    the batch needs serves many short sequences fastest.
    Returns out [batch, heads, d] bfloat16, or (out, lse [batch, heads]
    float32).  A head with nothing to attend to gives zeros and -inf.
    """
    if stream is None and out is None and out_lse is None and workspace is None:
        made = (_calls or _usual()).paged_attention(q, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, positions,
                                                    scale, return_lse)
        if made is not None:
            return _made(made, "paged_attention")
    dev = _device_of(q, "q")
    shape, strides = q.shape, q.stride()
    if q.dtype is not _BF16 or len(shape) != 3 or strides[2] != 1:
        _cuda_strided(q, "q", _BF16, 3)
    batch, heads, d = shape
    if heads > 1 and strides[1] != d:
        raise ValueError("the heads of q must be contiguous")
    kc, vc, (_, kv_heads, _, cache_d) = _two_caches(k_cache, v_cache, k_scale, v_scale, dev)
    if cache_d != d:
        raise ValueError("q and the caches disagree on d")
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError("heads must be a multiple of kv_heads")
    table_stride, width = _table(block_table, seq_lens, batch, dev)
    lists = c = 0
    if positions is not None:
        _cuda(positions, "positions", _I32)
        _same_device(q, positions=positions)
        if positions.dim() != 3 or positions.shape[0] != batch:
            raise ValueError("positions must be [batch, lists, c]")
        lists, c = positions.shape[1:]
        if lists < 1 or c < 1 or lists % kv_heads or heads % lists:
            raise ValueError("positions needs c >= 1 and lists a multiple of kv_heads that divides heads")
    _int32(heads=heads, lists=lists, c=c)
    _given_workspace(workspace, q)

    def body(out, out_lse, ws, sh):
        out = _out(out, shape, _BF16, "out", dev)
        if return_lse or out_lse is not None:
            out_lse = _out(out_lse, (batch, heads), _F32, "out_lse", dev)
        if ws is None:
            ws = _workspace(_workspace_bytes(paged_attention_workspace_bytes, 1, 1, 0, d), dev, sh)
        _check(load_library().paged_attention(
            q.data_ptr(), strides[0], batch, heads, ctypes.byref(kc), ctypes.byref(vc), block_table.data_ptr(),
            table_stride, width, seq_lens.data_ptr(), _pointer(positions), lists, c,
            d ** -0.5 if scale is None else scale, out.data_ptr(), _pointer(out_lse), ws.data_ptr(), _bytes(ws), sh),
            "paged_attention")
        return (out, out_lse) if return_lse else out

    return _on(dev, stream, body, out, out_lse, workspace)


def cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
                *, k_scale=None, v_scale=None, stream=None) -> None:
    """Write new tokens' keys and values into a paged cache, quantising them if it is e4m3.

    k, v: [tokens, kv_heads, d] bfloat16 (strides over tokens and heads are
    free: slices of a projection's output need no copy).  slots: [tokens] int64,
    page * page_size + offset; negative = not written.  The slots of one call
    must be distinct.  Caches and scales as in paged_attention; an e4m3 row
    gets the smallest power-of-two scale that holds it.
    """
    if stream is None:
        made = (_calls or _usual()).cache_write(k, v, k_cache, v_cache, slots, k_scale, v_scale)
        if made is not None:
            _made(made, "cache_write")
            return
    dev = _device_of(k, "k")
    kc, vc, cache_shape = _two_caches(k_cache, v_cache, k_scale, v_scale, dev)
    shape, ks = k.shape, k.stride()
    try:
        vs = v.stride()
        good = (k.dtype is _BF16 and v.dtype is _BF16 and len(shape) == 3 and ks[2] == 1 and vs[2] == 1
                and v.shape == shape and v.get_device() == dev and slots.get_device() == dev and slots.dtype is _I64
                and slots.shape == shape[:1] and slots.is_contiguous())
    except (AttributeError, TypeError, IndexError):
        good = False
    if not good:
        _cuda_strided(k, "k", _BF16, 3)
        _cuda_strided(v, "v", _BF16, 3)
        if v.shape != shape:
            raise ValueError("k and v must have the same shape")
        _cuda(slots, "slots", _I64)
        if slots.dim() != 1 or slots.numel() != shape[0]:
            raise ValueError("slots must be [tokens]")
        _same_device(k, v=v, slots=slots)
        vs = v.stride()
    if shape[1] != cache_shape[1] or shape[2] != cache_shape[3]:
        raise ValueError("k and v must be [tokens, kv_heads, d]")

    def body(sh):
        _check(load_library().cache_write(k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], shape[0],
                                          ctypes.byref(kc), ctypes.byref(vc), slots.data_ptr(), sh), "cache_write")

    _on(dev, stream, body)


def cache_read(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, n: int, *, scale=None,
               out=None, stream=None) -> torch.Tensor:
    """The first n tokens of every sequence as contiguous rows [batch, kv_heads, n, d] bfloat16.

    Rows behind a sequence's end are zeros.  `out.view(-1, n, d)` is the key
    matrix per row that score_topk and score_rerank take, for sequences of n
    tokens or more: a row of zeros scores 0, above every key of negative score.
    Sequences of unlike lengths take calls of their own, each with its length as n.
    """
    if stream is None and out is None:
        made = (_calls or _usual()).cache_read(cache, block_table, seq_lens, n, scale)
        if made is not None:
            return _made(made, "cache_read")
    dev = _device_of(cache, "cache")
    c, (_, kv_heads, _, d) = _cache(cache, scale, "cache", dev)
    batch = seq_lens.numel() if isinstance(seq_lens, torch.Tensor) else 0
    table_stride, width = _table(block_table, seq_lens, batch, dev)
    n = int(n)
    if out is not None and tuple(out.shape) != (batch, kv_heads, n, d):
        raise ValueError("out must be [batch, kv_heads, n, d]")

    def body(out, sh):
        out = _out(out, (batch, kv_heads, max(n, 0), d), _BF16, "out", dev)
        _check(load_library().cache_read(ctypes.byref(c), block_table.data_ptr(), table_stride, width,
                                         seq_lens.data_ptr(), batch, n, out.data_ptr() or None, sh), "cache_read")
        return out

    return _on(dev, stream, body, out)


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
    if stream is None and out_scores is None and out_parent is None and out_token is None and workspace is None:
        made = (_calls or _usual()).topk_beam(logits, beam_scores, k)
        if made is not None:
            return _made(made, "topk_beam")
    dev = _device_of(logits, "logits")
    bf16 = logits.dtype is _BF16
    try:
        good = ((bf16 or logits.dtype is _F32) and logits.dim() == 3 and logits.is_contiguous()
                and beam_scores.get_device() == dev and beam_scores.dtype is _F32
                and beam_scores.shape == logits.shape[:2] and beam_scores.is_contiguous())
    except (AttributeError, TypeError):
        good = False
    if not good:
        _cuda(logits, "logits", _BF16 if bf16 else _F32)
        _cuda(beam_scores, "beam_scores", _F32)
        if logits.dim() != 3 or tuple(beam_scores.shape) != tuple(logits.shape[:2]):
            raise ValueError("logits must be [batch, beams, n] and beam_scores [batch, beams]")
        _same_device(logits, beam_scores=beam_scores)
    _given_workspace(workspace, logits)
    batch, beams, n = logits.shape
    _int32(beams=beams, k=k)

    def body(out_scores, out_parent, out_token, ws, sh):
        shape = (batch, max(k, 0))
        out_scores = _out(out_scores, shape, _F32, "out_scores", dev)
        out_parent = _out(out_parent, shape, _I32, "out_parent", dev)
        out_token = _out(out_token, shape, _I32, "out_token", dev)
        if ws is None:
            ws = torch.empty(_workspace_bytes(topk_beam_workspace_bytes, batch, beams, n, k), dtype=torch.uint8,
                             device=_devices[dev])
        lib = load_library()
        fn = lib.topk_beam_bf16 if bf16 else lib.topk_beam
        _check(fn(logits.data_ptr(), beam_scores.data_ptr(), batch, beams, n, k, out_scores.data_ptr(),
                  out_parent.data_ptr(), out_token.data_ptr(), ws.data_ptr(), _bytes(ws), sh), "topk_beam")
        return out_scores, out_parent, out_token

    return _on(dev, stream, body, out_scores, out_parent, out_token, workspace)


def beam_reorder(states, parents: torch.Tensor, *, out=None, stream=None):
    """Per-beam states in the order topk_beam chose.

    states: a contiguous tensor [batch, beams, ...] of any dtype, or a list or
    tuple of up to 256 of them; parents: [batch, k] int32.  Returns the same
    with [batch, k, ...]: row (b, j) is row (b, parents[b, j]), zeros where
    that is -1.  `out` (of the same form) must not overlap the states.  Of a page
    table, rows of one parent name the same pages: of a page that is not full each
    needs a copy of its own before the next token is written into it.
    """
    one = isinstance(states, torch.Tensor)
    if stream is None and out is None:
        made = (_calls or _usual()).beam_reorder([states] if one else states, parents)
        if made is not None:
            made = _made(made, "beam_reorder")
            return made[0] if one else made
    src = [states] if one else list(states)
    dev = _device_of(parents, "parents")
    if parents.dtype is not _I32 or not parents.is_contiguous():
        _cuda(parents, "parents", _I32)
    if not src or parents.dim() != 2:
        raise ValueError("states needs a tensor at least and parents must be [batch, k]")
    batch, k = parents.shape
    beams = 0
    sizes = []
    for i, t in enumerate(src):
        if isinstance(t, torch.Tensor) and (t.is_conj() or t.is_neg()):  # bytes that stand for something else
            t = src[i] = t.resolve_conj().resolve_neg()
        if not isinstance(t, torch.Tensor) or t.get_device() != dev or not t.is_contiguous():
            _cuda(t, "states", t.dtype if isinstance(t, torch.Tensor) else None)
            _same_device(parents, states=t)
        shape = t.shape
        beams = beams or (shape[1] if len(shape) > 1 else 0)
        if len(shape) < 2 or shape[0] != batch or shape[1] != beams:
            raise ValueError("every state must be [batch, beams, ...]")
        n = t.numel()
        if n == 0:
            raise ValueError("states must not be empty")
        sizes.append(n // (batch * beams) * t.element_size())
    _int32(beams=beams, k=k)
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != len(src):
            raise ValueError("out needs one tensor per state")
        for t, o in zip(src, out):
            _cuda(o, "out", t.dtype)
            _same_device(parents, out=o)
            if o.is_conj() or o.is_neg():
                raise ValueError("out must not be a conjugate or negative view")
            if tuple(o.shape) != (batch, k) + tuple(t.shape[2:]):
                raise ValueError("out must be [batch, k, ...]")

    def body(dst, sh):
        if dst is None:
            dst = [t.new_empty((batch, k) + t.shape[2:]) if k != beams else torch.empty_like(t) for t in src]
        m = len(src)
        pointers = ctypes.c_void_p * m
        _check(load_library().beam_reorder(pointers(*[t.data_ptr() for t in src]), pointers(*[t.data_ptr() for t in dst]),
                                           (ctypes.c_int64 * m)(*sizes), m, batch, beams, k, parents.data_ptr(), sh),
               "beam_reorder")
        return dst[0] if one else dst

    return _on(dev, stream, body, out)
