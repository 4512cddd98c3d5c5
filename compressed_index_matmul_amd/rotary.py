"""Rotary positions of queries and keys, with norms of each head.

* :class:`Rotary`      -- the frequencies of a model's positions, on the GPU
* :func:`attn_rotate`  -- queries and keys to their positions, one launch

Tensors, streams and errors as in :mod:`.attention`.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from .attention import ATTN_HEAD_DIMS, _any_type, _array, _call, _heads, _ints
from .attention_abi import AttnRotary
from .streams import empty as _empty, resolve as _resolve

__all__ = ["Rotary", "attn_rotate"]


def _positive(scaling: dict, name: str, default=None) -> float:
    v = scaling.pop(name, default)
    if v is None:
        raise ValueError(f"scaling needs {name}")
    v = float(v)
    if not math.isfinite(v) or v <= 0.0:
        raise ValueError(f"scaling: {name} must be positive, got {v}")
    return v


def _frequencies(rot: int, base: float, scaling: Optional[dict]):
    """(angles a position of the rot / 2 pairs, gain)."""
    scaling = dict(scaling or {"kind": None})
    kind, gain = scaling.pop("kind", None), 1.0
    if kind not in (None, "linear", "base", "yarn", "bands"):
        raise ValueError(f"scaling kind must be linear, base, yarn or bands, got {kind!r}")
    factor = 1.0 if kind is None else _positive(scaling, "factor")
    if kind == "base":
        base *= factor ** (rot / max(rot - 2, 1))
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        freq = [w / factor for w in freq]
    elif kind == "yarn":
        original = _positive(scaling, "original")
        fast, slow = _positive(scaling, "beta_fast", 32.0), _positive(scaling, "beta_slow", 1.0)
        gain = _positive(scaling, "gain", max(0.1 * math.log(factor) + 1.0, 1.0))

        def pair_of(turns):  # the pair that makes so many turns over the original context
            return rot * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        low, high = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), rot - 1)
        for i, w in enumerate(freq):
            ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            freq[i] = w / factor * ramp + w * (1.0 - ramp)
    elif kind == "bands":
        original = _positive(scaling, "original")
        low, high = _positive(scaling, "low", 1.0), _positive(scaling, "high", 4.0)
        if high <= low:
            raise ValueError(f"scaling: high must be above low, got {low} and {high}")
        for i, w in enumerate(freq):
            keep = min(max((original * w / (2.0 * math.pi) - low) / (high - low), 0.0), 1.0)
            freq[i] = w / factor * (1.0 - keep) + w * keep
    if scaling:
        raise ValueError(f"scaling kind {kind!r} takes no {sorted(scaling)}")
    return freq, gain


class Rotary:
    """Frequencies of rotary positions for heads of head_dim (64, 128 or 256).

    The first rot_dim channels (a multiple of 16; default: all) turn in pairs
    (i, i + rot_dim / 2), or (2 i, 2 i + 1) with interleaved, by pos times
    base ** (-2 i / rot_dim).  scaling stretches them for long contexts:

    * ``{"kind": "linear", "factor": f}``: every frequency divided by f;
    * ``{"kind": "base", "factor": f}``: the base times f ** (R / (R - 2)), which
      divides the slowest frequency by f and leaves the fastest;
    * ``{"kind": "yarn", "factor": f, "original": n}``: divided by f for pairs of
      at most beta_slow (1) turns over the n positions of the original context,
      as they are from beta_fast (32) turns on, a ramp over the pairs between;
      sine and cosine times gain (default 0.1 log f + 1, and 1 up to f = 1);
    * ``{"kind": "bands", "factor": f, "original": n}``: the same by turns, from
      low (1) to high (4), with the ramp over the turns.

    inv_freq gives the rot_dim / 2 angles a position instead.  ``inv_freq``
    (Python floats), ``gain`` and ``turns`` (int64 on the device, 2^-64 of a turn a
    position) are the handle's state, ready for any stream once it is made."""

    def __init__(self, head_dim: int, rot_dim: Optional[int] = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[dict] = None, inv_freq: Optional[Sequence[float]] = None, device="cuda"):
        if head_dim not in ATTN_HEAD_DIMS:
            raise ValueError(f"head_dim must be one of {ATTN_HEAD_DIMS}, got {head_dim}")
        rot = head_dim if rot_dim is None else int(rot_dim)
        if rot < 16 or rot > head_dim or rot % 16:
            raise ValueError(f"rot_dim must be a multiple of 16 up to {head_dim}, got {rot}")
        base = float(base)
        if not math.isfinite(base) or base <= 1.0:
            raise ValueError(f"base must be above 1, got {base}")
        if inv_freq is not None:
            if scaling is not None:
                raise ValueError("inv_freq is taken as it is: scaling must be None")
            freq, gain = [float(w) for w in inv_freq], 1.0
            if len(freq) != rot // 2:
                raise ValueError(f"inv_freq must hold {rot // 2} angles, got {len(freq)}")
        else:
            freq, gain = _frequencies(rot, base, scaling)
        if not all(math.isfinite(w) for w in freq):
            raise ValueError("frequencies must be finite")
        self.head_dim, self.rot_dim, self.interleaved = head_dim, rot, bool(interleaved)
        self.inv_freq, self.gain = freq, gain
        turns = [round(math.ldexp(math.fmod(w / (2.0 * math.pi), 1.0), 64)) for w in freq]
        turns = [(t + 2**63) % 2**64 - 2**63 for t in turns]  # two's complement
        self.turns = torch.tensor(turns, dtype=torch.int64).to(device)
        self.device = self.turns.device
        self.desc = AttnRotary(head_dim, rot, int(self.interleaved), gain, self.turns.data_ptr())


def _weight(w, d: int, dev, name: str):
    if w is None:
        return None, None
    if not isinstance(w, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dt = _any_type(w.dtype, name)
    p = _array(w, (d,), w.dtype, dev, name)
    if p & 15:
        raise ValueError(f"{name} must start at a 16-byte boundary")
    return p, dt


def _result(out, shape, dtype, dev, st, name: str):
    if out is None:
        out = _empty(shape, dtype, dev, st)
        return out, out.data_ptr()
    p = _array(out, shape, dtype, dev, name)
    if p & 15:
        raise ValueError(f"{name} must start at a 16-byte boundary")
    return out, p


def attn_rotate(q, k, pos, rotary: Rotary, q_weight=None, k_weight=None, eps: float = 1e-6, dtype=None, out_q=None,
                out_k=None, stream=None):
    """Queries and keys to their positions, after a norm of each head where a
    weight is given: x / sqrt(mean(x^2) + eps) * weight.

    q [T, Hq, D] and k [T, Hk, D] (or None), float32, bfloat16 or float16, slices
    of one fused row or not; pos int32 [T]; q_weight and k_weight [D] of one type.
    Returns packed (q, k) of `dtype` (default: q's), q alone where k is None.
    out_q and out_k may be q and k themselves, where these are packed and of
    that type, and must not overlap the inputs otherwise."""
    if not isinstance(rotary, Rotary):
        raise TypeError("rotary must be a Rotary")
    hq_ = _heads(q, "q")
    dev = q.device
    t, hq, d = q.shape
    src = _any_type(q.dtype, "q")
    dtype = q.dtype if dtype is None else dtype
    dst = _any_type(dtype, "dtype")
    if d != rotary.head_dim:
        raise ValueError(f"q has heads of {d} channels, rotary is for {rotary.head_dim}")
    if rotary.device != dev:
        raise ValueError(f"rotary is on {rotary.device}; it must be on {dev}")
    if hq < 1:
        raise ValueError("q has no heads")
    hk, hk_ = 0, None
    if k is not None:
        hk_ = _heads(k, "k", dev)
        if k.dtype != q.dtype:
            raise TypeError(f"q is {q.dtype} and k is {k.dtype}; they must agree")
        hk = k.shape[1]
        if k.shape[0] != t or k.shape[2] != d or hk < 1:
            raise ValueError(f"k must be [{t}, heads, {d}], got {tuple(k.shape)}")
    elif k_weight is not None or out_k is not None:
        raise ValueError("k_weight and out_k need k")
    pp = _ints(pos, (t,), dev, "pos")
    qw, qt = _weight(q_weight, d, dev, "q_weight")
    kw, kt = _weight(k_weight, d, dev, "k_weight")
    if qt is not None and kt is not None and qt != kt:
        raise TypeError(f"q_weight is {q_weight.dtype} and k_weight is {k_weight.dtype}; they must agree")
    handle, st = _resolve(stream, dev)
    oq, pq = _result(out_q, (t, hq, d), dtype, dev, st, "out_q")
    ok, pk = _result(out_k, (t, hk, d), dtype, dev, st, "out_k") if hk else (None, None)
    _call("attn_rotate", dev, handle, rotary.desc, hq_, hk_, src, t, hq, hk, pp, qw, kw,
          next((x for x in (qt, kt) if x is not None), 0), float(eps), pq, pk, dst)
    return (oq, ok) if hk else oq
