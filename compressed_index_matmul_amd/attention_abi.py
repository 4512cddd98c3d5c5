"""The attention entry points' part of the C ABI (``include/vqmm.h``): element
type, mirrors of the structures, argument types.  Needs no torch, so that the
package loads the library without it."""
from __future__ import annotations

import ctypes

VQ_F16 = 2

_I32, _I64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class AttnHeads(ctypes.Structure):
    """Mirror of ``struct attn_heads``."""
    _fields_ = [("data", _P), ("token_stride", _I64), ("head_stride", _I64)]


class AttnBatch(ctypes.Structure):
    """Mirror of ``struct attn_batch``."""
    _fields_ = [("dtype", _I32), ("n_q_heads", _I32), ("n_kv_heads", _I32), ("head_dim", _I32), ("n_seqs", _I32),
                ("total_q", _I32), ("total_k", _I32), ("causal", _I32), ("scale", ctypes.c_float), ("reserved", _I32),
                ("cu_q", _P), ("cu_k", _P)]


class KV4CacheDesc(ctypes.Structure):
    """Mirror of ``struct kv4_cache``."""
    _fields_ = [("n_pages", _I32), ("page_size", _I32), ("n_kv_heads", _I32), ("head_dim", _I32), ("codes", _P),
                ("scales", _P), ("weights", _P), ("pos", _P)]


class KV4Seqs(ctypes.Structure):
    """Mirror of ``struct kv4_seqs``."""
    _fields_ = [("n_seqs", _I32), ("max_pages", _I32), ("block_table", _P), ("lens", _P)]


ATTN_EXPORTS = ("attn_prompt", "attn_prompt_workspace_size", "attn_prompt_weights",
                "attn_prompt_weights_workspace_size", "kv4_append", "kv4_read", "kv4_attend",
                "kv4_attend_workspace_size", "kv4_evict", "kv4_evict_workspace_size")


def declare(L) -> None:
    """Argument types of the attention entry points of the loaded library."""
    H, B, C, S = (ctypes.POINTER(t) for t in (AttnHeads, AttnBatch, KV4CacheDesc, KV4Seqs))
    z = ctypes.c_size_t
    for name, res, args in (
            ("attn_prompt", ctypes.c_int, [B, H, H, H, _P, _P, _P, z, _P]),
            ("attn_prompt_workspace_size", z, [B]),
            ("attn_prompt_weights", ctypes.c_int, [B, H, H, _P, _I32, _I32, _P, _P, z, _P]),
            ("attn_prompt_weights_workspace_size", z, [B, _I32]),
            ("kv4_append", ctypes.c_int, [C, S, H, H, _I32, _I32, _P, _P, _P, _P]),
            ("kv4_read", ctypes.c_int, [C, S, _P, _I32, _I32, _P, _P, _P]),
            ("kv4_attend", ctypes.c_int, [C, S, H, _I32, _I32, ctypes.c_float, _I32, _I32, _P, _P, _P, z, _P]),
            ("kv4_attend_workspace_size", z, [C, _I32, _I32, _I32, _I32]),
            ("kv4_evict", ctypes.c_int, [C, S, _P, _I32, _I32, _I32, _P, z, _P]),
            ("kv4_evict_workspace_size", z, [C, _I32, _I32, _I32])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
