"""Float64 oracle of the attention operators, in plain numpy.

Written from the definitions in ``include/vqmm.h``: attention over packed
prompts, the weights a prompt's keys gather, the 4-bit cache's encoding and
layout, single-token attention over it and eviction.  Nothing here imports
the package.

Each ``*_ref`` returns the exact result next to the scale that the fp32 and
16-bit roundings of the kernels are bounded by (see :func:`prompt_bound`).
"""
from __future__ import annotations

import numpy as np

GROUP = 32


def _visible(lq: int, lk: int, causal: bool) -> np.ndarray:
    """[lq, lk] truth values: the last query sees the last key."""
    if not causal:
        return np.ones((lq, lk), bool)
    return np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)


def softmax_rows(s: np.ndarray):
    """(probabilities, log sum of exponentials) of rows whose masked entries
    are -inf; a row of only masked entries gives zeros and -inf."""
    top = s.max(-1, keepdims=True) if s.shape[-1] else np.full(s.shape[:-1] + (1,), -np.inf)
    safe = np.where(np.isneginf(top), 0.0, top)
    e = np.exp(s - safe)
    l = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.log(l) + safe
    return e / np.where(l == 0, 1.0, l), lse[..., 0]


def prompt_ref(q, k, v, cu_q, cu_k, scale, causal):
    """q [Tq, Hq, D], k, v [Tk, Hkv, D] float64.  Returns out, lse [Hq, Tq],
    sum_j p_j |v_j| (out's scale), sum_j |v_j| and the largest scale *
    sum |q k| of each row [Hq, Tq]."""
    tq, hq, d = q.shape
    hkv = k.shape[1]
    out, mag, vsum = np.zeros((tq, hq, d)), np.zeros((tq, hq, d)), np.zeros((tq, hq, d))
    lse, smag = np.full((hq, tq), -np.inf), np.zeros((hq, tq))
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        see = _visible(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], causal)
        if see.size == 0:
            continue
        for h in range(hq):
            kk, vv = k[rk, h * hkv // hq], v[rk, h * hkv // hq]
            s = np.where(see, q[rq, h] @ kk.T * scale, -np.inf)
            p, lse[h, rq] = softmax_rows(s)
            out[rq, h] = p @ vv
            mag[rq, h] = p @ np.abs(vv)
            vsum[rq, h] = see @ np.abs(vv)
            smag[h, rq] = np.where(see, np.abs(q[rq, h]) @ np.abs(kk).T * scale, 0.0).max(-1)
    return out, lse, mag, vsum, smag


def prompt_weights_ref(q, k, lse, cu_q, cu_k, scale, causal, last):
    """[Hkv, Tk], and the largest scale * sum |q k| a key meets."""
    hq, hkv = q.shape[1], k.shape[1]
    out, smag = np.zeros((hkv, k.shape[0])), np.zeros((hkv, k.shape[0]))
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        rk = slice(cu_k[b], cu_k[b + 1])
        see = _visible(lq, lk, causal)
        if last:
            see[:max(0, lq - last)] = False
        if see.size == 0:
            continue
        for h in range(hq):
            qq, kk = q[cu_q[b]:cu_q[b + 1], h], k[rk, h * hkv // hq]
            norm = lse[h, cu_q[b]:cu_q[b + 1], None]
            arg = qq @ kk.T * scale - np.where(np.isneginf(norm), 0.0, norm)
            out[h * hkv // hq, rk] += np.where(see & ~np.isneginf(norm), np.exp(np.where(see, arg, 0.0)), 0.0).sum(0)
            m = np.where(see, np.abs(qq) @ np.abs(kk).T * scale, 0.0).max(0)
            smag[h * hkv // hq, rk] = np.maximum(smag[h * hkv // hq, rk], m)
    return out, smag


# Largest relative error of one rounding: bf16 keeps 8 significant bits, fp16 11.
ROUND = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def prompt_bound(out, mag, vsum, smag, d, n, kind, p_kind=None, v_round=0.0):
    """Largest |error| of a kernel's output of 16-bit type `kind`.

    A score is an fp32 sum of d exact products (off by d 2^-24 of their
    magnitudes), times scale log2(e) in fp32 (2^-22 of itself); exp2 and the sum of
    n terms add (n + 4) 2^-24.  Twice that, for numerator and sum, is the
    relative error of a probability, which is then rounded to 16 bits.  fp16
    ones are taken so that the largest is 2^7 at least: below fp16's normal
    range they are off by 2^-25, 2^-32 of the largest, which is at most one, so
    by 2^-32 of each |v|.  Values may carry v_round; the result is rounded
    once."""
    s = np.swapaxes(smag, 0, 1)[:, :, None]
    delta = 2.0 * (s * (d + 8) * 2.0 ** -24 + s * 2.0 ** -22 + (n + 4) * 2.0 ** -24)
    err = (delta + ROUND[p_kind or kind] + v_round) * 1.01 * mag + 2.0 ** -32 * vsum
    return err + ROUND[kind] * 1.01 * (np.abs(out) + err) + 2.0 ** -25


def lse_bound(lse, smag, d, n):
    """The scores' error, that of the sum and of its logarithm."""
    with np.errstate(invalid="ignore"):
        return smag * ((d + 8) * 2.0 ** -24 + 2.0 ** -22) + (n + 4) * 2.0 ** -24 + np.where(
            np.isfinite(lse), np.abs(lse), 0.0) * 2.0 ** -22 + 2.0 ** -22


# ---------------------------------------------------------------------------
# the 4-bit cache
# ---------------------------------------------------------------------------
def kv4_encode(x: np.ndarray):
    """Codes [..., D] uint8, steps and minima [..., D / 32] float16 of float32
    values, each step one float32 operation."""
    f = np.float32
    x = np.asarray(x, f)
    with np.errstate(invalid="ignore"):
        x = np.where(np.isnan(x), x, np.clip(x, f(-32768), f(32768))).astype(f)
        g = x.reshape(*x.shape[:-1], -1, GROUP)
        low, high = g.min(-1), g.max(-1)
        m = low.astype(np.float16)
        s = ((high - low) * (f(1) / f(15))).astype(np.float16)
        sf = s.astype(f)
        r = np.where(sf > 0, f(1) / np.where(sf > 0, sf, f(1)), f(0)).astype(f)
        t = (g - m.astype(f)[..., None]) * r[..., None]
        c = np.clip(np.rint(t), 0, 15)
    return np.where(np.isnan(c), 0, c).astype(np.uint8).reshape(x.shape), s, m


def kv4_values(c, s, m) -> np.ndarray:
    """What codes stand for, float64."""
    g = c.reshape(*c.shape[:-1], -1, GROUP).astype(np.float64)
    return (g * s.astype(np.float64)[..., None] + m.astype(np.float64)[..., None]).reshape(c.shape)


class Pool:
    """A cache pool as numpy arrays, addressed slot by slot from the layout's
    description."""

    def __init__(self, codes, scales, weights, pos):
        self.codes, self.scales, self.weights, self.pos = codes, scales, weights, pos
        self.page, self.d = weights.shape[2], scales.shape[4] * GROUP
        c = np.arange(self.d)
        octet = c // 8
        word = (octet % 4) * (self.d // GROUP) + octet // 4
        self.key_byte, self.shift = word * 4 + (c % 8) // 2, 4 * (c % 2)
        self.value_byte = c // 2 * 4

    def _bytes(self, kind, h, page, at):
        if kind == 0:
            return at * (self.d // 2) + self.key_byte
        return at // 4 * (2 * self.d) + self.value_byte + (0, 2, 1, 3)[at % 4]

    def get(self, kind, h, page, at):
        """Codes, steps and minima of one slot."""
        c = (self.codes[page, kind, h][self._bytes(kind, h, page, at)] >> self.shift) & 15
        g = self.scales[page, kind, h, at // 4]
        return c, g[:, at % 4], g[:, 4 + at % 4]

    def put(self, kind, h, page, at, c, s, m):
        raw, where = self.codes[page, kind, h], self._bytes(kind, h, page, at)
        raw[where[0::2]] = c[0::2] | (c[1::2] << 4)
        g = self.scales[page, kind, h, at // 4]
        g[:, at % 4], g[:, 4 + at % 4] = s, m

    def values(self, kind, h, table, n):
        """float64 [n, D] of a sequence's first n slots."""
        out = np.zeros((n, self.d))
        for i in range(n):
            out[i] = kv4_values(*self.get(kind, h, table[i // self.page], i % self.page))
        return out

    def append(self, k, v, cu, table, start, pos=None, weights=None):
        """k, v [T, Hkv, D] float32 values."""
        enc = [kv4_encode(x) for x in (k, v)]
        for b in range(len(cu) - 1):
            for i in range(cu[b + 1] - cu[b]):
                slot, row = start[b] + i, cu[b] + i
                if slot >= table.shape[1] * self.page:
                    break
                page, at = table[b, slot // self.page], slot % self.page
                for h in range(k.shape[1]):
                    for kind, (c, s, m) in enumerate(enc):
                        self.put(kind, h, page, at, c[row, h], s[row, h], m[row, h])
                    self.weights[page, h, at] = 0.0 if weights is None else weights[h, row]
                    self.pos[page, h, at] = (start[b] if pos is None else pos[b]) + i

    def evict(self, table, lens, next_pos, keep, recent):
        for b, n in enumerate(lens):
            if n <= keep:
                continue
            slots = np.arange(n)
            pages, at = table[b, slots // self.page], slots % self.page
            for h in range(self.weights.shape[1]):
                w = self.weights[pages, h, at].astype(np.float64)
                free = self.pos[pages, h, at] < int(next_pos[b]) - recent  # not protected
                lowest = free & np.isnan(w)
                order = np.lexsort((slots, np.where(free & ~lowest, -w, 0.0), lowest, free))
                stays = np.zeros(n, bool)
                stays[order[:keep]] = True
                for dst, src in zip(slots[~stays & (slots < keep)], slots[stays & (slots >= keep)]):
                    for kind in (0, 1):
                        self.put(kind, h, pages[dst], at[dst], *self.get(kind, h, pages[src], at[src]))
                    self.weights[pages[dst], h, at[dst]] = self.weights[pages[src], h, at[src]]
                    self.pos[pages[dst], h, at[dst]] = self.pos[pages[src], h, at[src]]


def attend_ref(q, pool: Pool, table, lens, scale):
    """q [B, Hq, D] float64.  Returns out, lse [B, Hq], p [list of [Hq, n]],
    out's scales (as prompt_ref) and the scores' scale, which counts steps
    and minima apart: scale * sum_g (s_g |q| . c + |m_g| sum |q|)."""
    bsz, hq, d = q.shape
    hkv = pool.weights.shape[1]
    out, mag, vsum = np.zeros((bsz, hq, d)), np.zeros((bsz, hq, d)), np.zeros((bsz, hq, d))
    lse, smag, probs = np.full((bsz, hq), -np.inf), np.zeros((bsz, hq)), []
    for b, n in enumerate(lens):
        probs.append(np.zeros((hq, n)))
        if n == 0:
            continue
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            kk, vv = pool.values(0, h, table[b], n), pool.values(1, h, table[b], n)
            parts = np.zeros((n, d))
            for i in range(n):
                c, s, m = pool.get(0, h, table[b, i // pool.page], i % pool.page)
                parts[i] = np.abs(s.astype(np.float64)).repeat(GROUP) * c + np.abs(m.astype(np.float64)).repeat(GROUP)
            p, lse[b, heads] = softmax_rows(q[b, heads] @ kk.T * scale)
            probs[b][heads] = p
            out[b, heads], mag[b, heads], vsum[b, heads] = p @ vv, p @ np.abs(vv), np.abs(vv).sum(0)
            smag[b, heads] = (np.abs(q[b, heads]) @ parts.T * scale).max(-1)
    return out, lse, probs, mag, vsum, smag
