"""Attention over packed prompts, the 4-bit key/value cache and eviction from it.

Argument marshalling for the attention entry points of ``include/vqmm.h``;
the package re-exports everything here.

* :func:`attn_prompt`         -- attention over packed prompts, grouped heads
* :func:`attn_prompt_weights` -- the attention weight each key gathers
* :class:`KV4Cache`           -- a pool of pages of 4-bit keys and values
* :func:`kv4_append`, :func:`kv4_read` -- packed rows into the cache and back
* :func:`kv4_attend`          -- one query a sequence against the cache
* :func:`kv4_attend_chunk`    -- several queries a sequence against it
* :func:`kv4_evict`           -- cut sequences down by accumulated weight

Tensors of heads are ``[tokens, heads, head_dim]`` with contiguous channels;
tokens and heads may be strided (slices of a fused row).  Offsets, lengths and
block tables are int32 device tensors; their contents are not read on the
host.  Sequence lengths in the cache are the caller's: ``kv4_append`` does not
raise them and ``kv4_evict`` does not lower them.

Every tensor has to be on one GPU.  ``stream`` (a torch stream or a raw handle;
default: the device's current stream) is where the work is enqueued.  What a
call allocates itself comes from that stream's memory, and what it returns may
be used on the caller's current stream too, once that has waited for `stream`.
Inputs made on another stream are the caller's to synchronise, as for any torch
operation.
"""

from __future__ import annotations

from typing import Optional

import torch

from .attention_abi import (ATTN_EXPORTS, VQ_F16, AttnBatch, AttnHeads, KV4CacheDesc, KV4Seqs,  # noqa: F401
                            declare)
from .streams import empty as _empty, resolve as _resolve

__all__ = ["VQ_F16", "KV4Cache", "attn_prompt", "attn_prompt_weights", "kv4_append", "kv4_read", "kv4_attend",
           "kv4_attend_workspace_size", "kv4_attend_chunk", "kv4_attend_chunk_workspace_size", "kv4_evict",
           "kv4_evict_workspace_size"]

KV4_GROUP = 32  # channels that share a step and a minimum
ATTN_HEAD_DIMS = (64, 128, 256)


def _pkg():
    import compressed_index_matmul_amd as m
    return m


_FN = {}

# The current device without building Python objects; the public call where
# this torch has no such name.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _fn(name):
    f = _FN.get(name)
    if f is None:
        f = _FN[name] = getattr(_pkg().lib(), name)
    return f


def _call(name, dev, handle, *args):
    """One library call on the stream `handle` with `dev` current."""
    fn = _FN.get(name) or _fn(name)
    if _current_device() == dev.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != 0:
        raise _pkg().VQError(status, name)


_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: VQ_F16}


def _half(t, name: str) -> int:
    v = _TYPES.get(t.dtype, 0)
    if not v:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return v


def _any_type(dtype, name: str) -> int:
    v = _TYPES.get(dtype)
    if v is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return v


def _heads(t, name: str, dev=None) -> AttnHeads:
    """[tokens, heads, head_dim] on the GPU `dev` (any, when None)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected [tokens, heads, head_dim]")
    if not t.is_cuda or (dev is not None and t.device != dev):
        raise ValueError(f"{name} is on {t.device}; it must be on {dev or 'a GPU'}")
    n, h, d = t.shape
    ts, hs, cs = t.stride()
    if cs != 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    if n <= 1:
        ts = h * d  # the stride of a single row has no meaning
    if h <= 1:
        hs = d
    if ts < 8 or hs < 8 or (ts | hs) & 7 or ts >= 1 << 22:
        raise ValueError(f"{name}: strides {t.stride()} must be positive multiples of 8, between tokens below 2^22")
    p = t.data_ptr()
    if p & 15:
        raise ValueError(f"{name} must start at a 16-byte boundary")
    return AttnHeads(p, ts, hs)


def _array(t, shape, dtype, dev, name: str) -> int:
    """Address of a contiguous tensor of the shape and type on the GPU `dev`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on {dev}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    return t.data_ptr()


def _ints(t, shape, dev, name: str) -> int:
    return _array(t, shape, torch.int32, dev, name)


def _output(out, like, dev, st):
    """`out`, checked, or a new tensor of `like`'s shape and type; its address."""
    if out is not None:
        return out, _array(out, like.shape, like.dtype, dev, "out")
    out = _empty(like.shape, like.dtype, dev, st)
    return out, out.data_ptr()


def _batch(q, k, cu_q, cu_k, scale, causal):
    dtype = _half(q, "q")
    if k.dtype != q.dtype:
        raise TypeError(f"q is {q.dtype} and k is {k.dtype}; they must agree")
    tq, hq, d = q.shape
    tk, hkv, dk = k.shape
    if d not in ATTN_HEAD_DIMS or dk != d:
        raise ValueError(f"head_dim must be one of {ATTN_HEAD_DIMS} and the same for q and k, got {d} and {dk}")
    if hkv < 1 or hq < 1 or hq % hkv:
        raise ValueError(f"{hq} query heads are no multiple of {hkv} key/value heads")
    dev = q.device
    if not isinstance(cu_q, torch.Tensor):
        raise TypeError("cu_q must be a torch tensor")
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [sequences + 1]")
    n = cu_q.numel() - 1
    pq = _ints(cu_q, (n + 1,), dev, "cu_q")
    pk = pq if cu_k is None else _ints(cu_k, (n + 1,), dev, "cu_k")
    if cu_k is None and tk != tq:
        raise ValueError(f"q has {tq} rows and k {tk}: pass cu_k")
    return AttnBatch(dtype, hq, hkv, d, n, tq, tk, int(bool(causal)), d ** -0.5 if scale is None else float(scale), 0,
                     pq, pk)


def _window(window, sinks):
    """(window, 0 for none; sinks) as the library takes them."""
    sinks = int(sinks)
    if window is None:
        if sinks:
            raise ValueError("sinks need a window")
        return 0, 0
    window = int(window)
    if window < 1 or sinks < 0:
        raise ValueError(f"window must be at least 1 and sinks not negative, got window={window} sinks={sinks}")
    return min(window, 2**31 - 1), min(sinks, 2**31 - 1)


def attn_prompt(q, k, v, cu_q, cu_k=None, scale: Optional[float] = None, causal: bool = True, out=None,
                return_lse: bool = False, workspace=None, stream=None, window: Optional[int] = None, sinks: int = 0):
    """softmax(scale q k^T) v over packed sequences.

    q [Tq, Hq, D], k and v [Tk, Hkv, D], bfloat16 or float16, Hq a multiple of
    Hkv, D 64, 128 or 256; cu_q (and cu_k, where the keys are packed
    differently: a chunk against its prefix) int32 [sequences + 1] offsets.
    causal: query i of Lq sees keys j <= i + Lk - Lq.  A query that sees no key
    gives zeros (lse -inf).  window (with causal): of these, only the newest
    `window` and the sequence's first `sinks`.  workspace: a device tensor (None
    allocates what the call needs; fewer rows may need more).  Returns out [Tq,
    Hq, D], with return_lse also the scores' log sum of exponentials, float32
    [Hq, Tq]."""
    hq_ = _heads(q, "q")
    dev = q.device
    hk, hv = _heads(k, "k", dev), _heads(v, "v", dev)
    b = _batch(q, k, cu_q, cu_k, scale, causal)
    if v.dtype != q.dtype or v.shape != k.shape:
        raise ValueError(f"v must be {q.dtype} {tuple(k.shape)}, got {v.dtype} {tuple(v.shape)}")
    if b.n_seqs == 0 and b.total_q:
        raise ValueError("rows without a sequence")
    window, sinks = _window(window, sinks)
    if window and not b.causal:
        raise ValueError("a window needs causal=True")
    name, more = ("attn_prompt_window", (window, sinks)) if window else ("attn_prompt", ())
    handle, st = _resolve(stream, dev)
    out, po = _output(out, q, dev, st)
    lse = _empty((b.n_q_heads, b.total_q), torch.float32, dev, st) if return_lse else None
    ws, pw, wb = _workspace(workspace, _fn(name + "_workspace_size")(b, *more) if workspace is None else 0, dev, st)
    _call(name, dev, handle, b, *more, hq_, hk, hv, po, None if lse is None else lse.data_ptr(), pw, wb)
    return (out, lse) if return_lse else out


def attn_prompt_weights(q, k, lse, cu_q, cu_k=None, scale: Optional[float] = None, causal: bool = True, last: int = 0,
                        out=None, accumulate: bool = False, workspace=None, stream=None):
    """The attention weight every key gathers: float32 [Hkv, Tk], summed over
    the heads of its group and over the last `last` queries of its sequence (0:
    all).  q, k, cu_q, cu_k, scale, causal and lse as attn_prompt takes and
    gives them; accumulate adds to `out` instead of writing it; workspace as
    for attn_prompt."""
    hq_ = _heads(q, "q")
    dev = q.device
    hk = _heads(k, "k", dev)
    b = _batch(q, k, cu_q, cu_k, scale, causal)
    pl = _array(lse, (b.n_q_heads, b.total_q), torch.float32, dev, "lse")
    last = int(last)
    if last < 0:
        raise ValueError(f"last must not be negative, got {last}")
    if b.n_seqs == 0 and b.total_k:
        raise ValueError("rows without a sequence")
    shape = (b.n_kv_heads, b.total_k)
    handle, st = _resolve(stream, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _empty(shape, torch.float32, dev, st)
    po = _array(out, shape, torch.float32, dev, "out")
    last = min(last, 2**31 - 1)
    ws, pw, wb = _workspace(workspace, _fn("attn_prompt_weights_workspace_size")(b, last) if workspace is None else 0, dev, st)
    _call("attn_prompt_weights", dev, handle, b, hq_, hk, pl, last, int(bool(accumulate)), po, pw, wb)
    return out


class KV4Cache:
    """A pool of pages of 4-bit keys and values, 5 bits a value with the steps
    and minima of its groups of 32 channels, and of each slot's accumulated
    attention weight and position.  ``page_size`` slots a page (a multiple of
    32, at most 1024).  The layout of ``codes``, ``scales``, ``weights`` and ``pos``
    is the C header's."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda"):
        if n_pages < 1 or n_kv_heads < 1 or page_size < 32 or page_size > 1024 or page_size % 32:
            raise ValueError(f"invalid cache: {n_pages} pages of {page_size} slots, {n_kv_heads} heads (page_size is a "
                             "multiple of 32 up to 1024)")
        if head_dim not in ATTN_HEAD_DIMS:
            raise ValueError(f"head_dim must be one of {ATTN_HEAD_DIMS}, got {head_dim}")
        dg = head_dim // KV4_GROUP
        self._set(torch.zeros((n_pages, 2, n_kv_heads, page_size * head_dim // 2), dtype=torch.uint8, device=device),
                  torch.zeros((n_pages, 2, n_kv_heads, page_size // 4, dg, 8), dtype=torch.float16, device=device),
                  torch.zeros((n_pages, n_kv_heads, page_size), dtype=torch.float32, device=device),
                  torch.zeros((n_pages, n_kv_heads, page_size), dtype=torch.int32, device=device))

    @classmethod
    def from_buffers(cls, codes, scales, weights, pos) -> "KV4Cache":
        """A cache over existing tensors of the documented shapes (not copied)."""
        self = cls.__new__(cls)
        self._set(codes, scales, weights, pos)
        return self

    def _set(self, codes, scales, weights, pos):
        if not all(isinstance(t, torch.Tensor) for t in (codes, scales, weights, pos)):
            raise TypeError("codes, scales, weights and pos must be torch tensors")
        if weights.dim() != 3 or scales.dim() != 6:
            raise ValueError("weights must be [pages, heads, slots] and scales [pages, 2, heads, slots / 4, groups, 8]")
        n, h, ps = weights.shape
        d = scales.shape[4] * KV4_GROUP
        if n < 1 or h < 1 or ps < 32 or ps > 1024 or ps % 32 or d not in ATTN_HEAD_DIMS:
            raise ValueError(f"invalid cache: {n} pages of {ps} slots, {h} heads of {d} channels")
        dev = weights.device
        pc = _array(codes, (n, 2, h, ps * d // 2), torch.uint8, dev, "codes")
        sc = _array(scales, (n, 2, h, ps // 4, d // KV4_GROUP, 8), torch.float16, dev, "scales")
        pw = _array(weights, (n, h, ps), torch.float32, dev, "weights")
        pp = _array(pos, (n, h, ps), torch.int32, dev, "pos")
        for p, name in ((pc, "codes"), (sc, "scales"), (pw, "weights"), (pp, "pos")):
            if p % 16:
                raise ValueError(f"{name} must start at a 16-byte boundary")
        self.codes, self.scales, self.weights, self.pos = codes, scales, weights, pos
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, self.device = n, ps, h, d, dev
        self.desc = KV4CacheDesc(n, ps, h, d, pc, sc, pw, pp)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.scales, self.weights, self.pos))


def _seqs(cache: KV4Cache, block_table, lens, name: str) -> KV4Seqs:
    dev = cache.device
    if dev.type != "cuda":
        raise ValueError(f"the cache is on {dev}; the kernels need it on a GPU")
    if not isinstance(block_table, torch.Tensor):
        raise TypeError("block_table must be a torch tensor")
    if block_table.dim() != 2 or block_table.shape[1] < 1:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}; expected [sequences, pages]")
    n, mp = block_table.shape
    return KV4Seqs(n, mp, _ints(block_table, (n, mp), dev, "block_table"),
                   None if lens is None else _ints(lens, (n,), dev, name))


def kv4_append(cache: KV4Cache, k, v, cu, block_table, start=None, pos=None, weights=None, stream=None) -> None:
    """Store packed rows k, v [T, Hkv, D] (float32, bfloat16 or float16): row
    cu[b] + i goes to slot start[b] + i of sequence b (start None: from 0).

    cu int32 [sequences + 1], block_table int32 [sequences, pages], start
    int32 [sequences]; pos int32 [sequences], the position of each sequence's
    first row (None: its slot); weights float32 [Hkv, T], the slots' accumulated
    weight so far (None: 0).  The caller raises the lengths.  A page that is
    written to must belong to one sequence of the table."""
    s = _seqs(cache, block_table, start, "start")
    dev = cache.device
    hk, hv = _heads(k, "k", dev), _heads(v, "v", dev)
    t = k.shape[0]
    if tuple(k.shape) != (t, cache.n_kv_heads, cache.head_dim) or v.shape != k.shape:
        raise ValueError(f"k and v must be [rows, {cache.n_kv_heads}, {cache.head_dim}], got {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    if v.dtype != k.dtype:
        raise TypeError(f"k is {k.dtype} and v is {v.dtype}; they must agree")
    dtype = _any_type(k.dtype, "k and v")
    pc = _ints(cu, (s.n_seqs + 1,), dev, "cu")
    pp = None if pos is None else _ints(pos, (s.n_seqs,), dev, "pos")
    pw = None if weights is None else _array(weights, (cache.n_kv_heads, t), torch.float32, dev, "weights")
    _call("kv4_append", dev, _resolve(stream, dev)[0], cache.desc, s, hk, hv, dtype, t, pc, pp, pw)


def kv4_read(cache: KV4Cache, cu, block_table, total: int, start=None, dtype=None, stream=None):
    """Slots start[b] + i of every sequence as packed rows: (k, v), each
    [total, Hkv, D] of dtype (bfloat16 by default).  total is cu's last entry
    (rows beyond cu are left as allocated)."""
    s = _seqs(cache, block_table, start, "start")
    dev = cache.device
    dtype = torch.bfloat16 if dtype is None else dtype
    dt = _any_type(dtype, "dtype")
    total = int(total)
    if total < 0:
        raise ValueError(f"total must not be negative, got {total}")
    pc = _ints(cu, (s.n_seqs + 1,), dev, "cu")
    shape = (total, cache.n_kv_heads, cache.head_dim)
    handle, st = _resolve(stream, dev)
    k, v = _empty(shape, dtype, dev, st), _empty(shape, dtype, dev, st)
    _call("kv4_read", dev, handle, cache.desc, s, pc, total, dt, k.data_ptr(), v.data_ptr())
    return k, v


def kv4_attend_workspace_size(cache: KV4Cache, n_seqs: int, n_q_heads: int, max_len: int, add_weights: bool = False) -> int:
    """Bytes of workspace kv4_attend needs."""
    return _fn("kv4_attend_workspace_size")(cache.desc, n_seqs, n_q_heads, max_len, int(bool(add_weights)))


def _workspace(workspace, need: int, dev, st):
    """The workspace (to be held until the call is queued), its address and size."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _empty((need,), torch.uint8, dev, st, returned=False)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch tensor")
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def kv4_attend(q, cache: KV4Cache, block_table, lens, scale: Optional[float] = None, max_len: Optional[int] = None,
               add_weights: bool = False, out=None, return_lse: bool = False, workspace=None, stream=None):
    """One query a sequence, q [sequences, Hq, D] bfloat16 or float16, over the
    first lens[b] slots of the cache.

    max_len: the host's bound on lens (longer ones count as max_len; default:
    the block table's capacity); a close one saves launch width and workspace.
    add_weights adds every slot's attention weight, summed over the heads of
    its group, to cache.weights; the pages must then not be shared between
    sequences (otherwise they may).  workspace: a device tensor of at least
    kv4_attend_workspace_size bytes (None allocates).  Returns out, with
    return_lse also float32 [sequences, Hq].  An empty sequence gives zeros
    and -inf."""
    s = _seqs(cache, block_table, lens, "lens")
    if lens is None:
        raise ValueError("kv4_attend needs lens")
    dev = cache.device
    hq_ = _heads(q, "q", dev)
    n, hq, d = q.shape
    if n != s.n_seqs or d != cache.head_dim or hq < 1 or hq % cache.n_kv_heads:
        raise ValueError(f"q must be [{s.n_seqs}, a multiple of {cache.n_kv_heads}, {cache.head_dim}], got {tuple(q.shape)}")
    dtype = _half(q, "q")
    capacity = s.max_pages * cache.page_size
    max_len = capacity if max_len is None else int(max_len)
    if max_len < 0:
        raise ValueError(f"max_len must not be negative, got {max_len}")
    max_len = min(max_len, capacity)
    handle, st = _resolve(stream, dev)
    out, po = _output(out, q, dev, st)
    lse = _empty((n, hq), torch.float32, dev, st) if return_lse else None
    weigh = int(bool(add_weights))
    ws, pw, wb = _workspace(workspace, kv4_attend_workspace_size(cache, n, hq, max_len, weigh) if workspace is None else 0,
                            dev, st)
    _call("kv4_attend", dev, handle, cache.desc, s, hq_, dtype, hq, d ** -0.5 if scale is None else float(scale),
          max_len, weigh, po, None if lse is None else lse.data_ptr(), pw, wb)
    return (out, lse) if return_lse else out


def kv4_attend_chunk_workspace_size(cache: KV4Cache, n_seqs: int, n_q_heads: int, total_q: int, max_len: int,
                                    max_q: Optional[int] = None, window: Optional[int] = None, sinks: int = 0) -> int:
    """Bytes of workspace that serve kv4_attend_chunk for these sizes and for
    smaller ones, window and sinks being the same (max_q None: total_q)."""
    return _fn("kv4_attend_chunk_workspace_size")(cache.desc, n_seqs, n_q_heads, total_q, *_window(window, sinks), max_len,
                                                  total_q if max_q is None else max_q)


def kv4_attend_chunk(q, cache: KV4Cache, block_table, lens, cu_q=None, scale: Optional[float] = None,
                     window: Optional[int] = None, sinks: int = 0, max_len: Optional[int] = None,
                     max_q: Optional[int] = None, out=None, return_lse: bool = False, workspace=None, stream=None):
    """Packed queries q [Tq, Hq, D], bfloat16 or float16, over the first lens[b]
    slots of their sequence, the last of which are the queries' own tokens
    (kv4_append them first, then raise lens): query i of Lq sees the slots up to
    i + lens[b] - Lq, under a window only the newest `window` of these and the
    sequence's first `sinks`.

    cu_q: int32 [sequences + 1] offsets (None: one query a sequence).  Windows
    count slots: the newest tokens, unless the sequence has been evicted from.
    max_len: the host's bound on lens (longer ones count as max_len; default:
    the block table's capacity); max_q: its bound on the queries of a sequence
    (default: Tq), which chooses how the work is cut.  workspace: a device tensor
    of at least kv4_attend_chunk_workspace_size bytes, of these sizes or of the
    largest call's (None allocates).  Returns out [Tq, Hq, D], with return_lse
    also float32 [Hq, Tq].  A query that sees nothing gives zeros and -inf."""
    s = _seqs(cache, block_table, lens, "lens")
    if lens is None:
        raise ValueError("kv4_attend_chunk needs lens")
    dev = cache.device
    hq_ = _heads(q, "q", dev)
    tq, hq, d = q.shape
    if d != cache.head_dim or hq < 1 or hq % cache.n_kv_heads:
        raise ValueError(f"q must be [queries, a multiple of {cache.n_kv_heads}, {cache.head_dim}], got {tuple(q.shape)}")
    dtype = _half(q, "q")
    if cu_q is None and tq != s.n_seqs:
        raise ValueError(f"{tq} queries for {s.n_seqs} sequences: pass cu_q")
    if s.n_seqs == 0 and tq:
        raise ValueError("rows without a sequence")
    pc = None if cu_q is None else _ints(cu_q, (s.n_seqs + 1,), dev, "cu_q")
    window, sinks = _window(window, sinks)
    capacity = s.max_pages * cache.page_size
    max_len = capacity if max_len is None else int(max_len)
    max_q = (1 if cu_q is None else tq) if max_q is None else int(max_q)
    if max_len < 0 or max_q < 0:
        raise ValueError(f"max_len and max_q must not be negative, got {max_len} and {max_q}")
    sizes = window, sinks, min(max_len, capacity), min(max_q, tq)
    handle, st = _resolve(stream, dev)
    out, po = _output(out, q, dev, st)
    lse = _empty((hq, tq), torch.float32, dev, st) if return_lse else None
    need = _fn("kv4_attend_chunk_workspace_size")(cache.desc, s.n_seqs, hq, tq, *sizes) if workspace is None else 0
    ws, pw, wb = _workspace(workspace, need, dev, st)
    _call("kv4_attend_chunk", dev, handle, cache.desc, s, hq_, dtype, hq, tq, pc, d ** -0.5 if scale is None else float(scale),
          *sizes, po, None if lse is None else lse.data_ptr(), pw, wb)
    return (out, lse) if return_lse else out


def kv4_evict_workspace_size(cache: KV4Cache, n_seqs: int, keep: int, max_len: int) -> int:
    """Bytes of workspace kv4_evict needs."""
    return _fn("kv4_evict_workspace_size")(cache.desc, n_seqs, keep, max_len)


def kv4_evict(cache: KV4Cache, block_table, lens, next_pos, keep: int, recent: int, max_len: Optional[int] = None,
              workspace=None, stream=None) -> None:
    """Cut every sequence longer than `keep` down to keep slots, each key/value
    head on its own: kept are the slots with pos >= next_pos[b] - recent, then
    those of the largest cache.weights.  Kept slots at or above keep move into
    the free ones below: every page of a sequence that is cut must belong to it
    alone (copy a shared prefix first).  lens and next_pos (the position of the next token)
    are int32 [sequences]; the caller then lowers lens to min(lens, keep)."""
    s = _seqs(cache, block_table, lens, "lens")
    if lens is None:
        raise ValueError("kv4_evict needs lens")
    dev = cache.device
    keep, recent = int(keep), int(recent)
    if keep < 1 or not 0 <= recent <= keep:
        raise ValueError(f"keep must be at least 1 and recent within 0..keep, got keep={keep} recent={recent}")
    capacity = s.max_pages * cache.page_size
    max_len = capacity if max_len is None else int(max_len)
    if max_len < 0:
        raise ValueError(f"max_len must not be negative, got {max_len}")
    max_len = min(max_len, capacity)
    pn = _ints(next_pos, (s.n_seqs,), dev, "next_pos")
    handle, st = _resolve(stream, dev)
    ws, pw, wb = _workspace(workspace, kv4_evict_workspace_size(cache, s.n_seqs, keep, max_len) if workspace is None else 0,
                            dev, st)
    _call("kv4_evict", dev, handle, cache.desc, s, pn, min(keep, 2**31 - 1), min(recent, 2**31 - 1), max_len, pw, wb)
