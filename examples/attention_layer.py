"""The attention half of one decoder layer on compressed weights: prompts,
then single tokens, over a 4-bit cache that is kept to a budget.

    python examples/attention_layer.py [--steps N] [--keep N] [--seed N]

The q/k/v and output projections are 2-stage 12-bit codebook weights
(SmolLM-135M's shape: rows of 576, 9 query and 3 key/value heads of 64); all
weights and inputs are synthetic.  A prompt goes through

    vq_gemm -> rotary positions -> attn_prompt -> vq_gemm
                                -> attn_prompt_weights -> kv4_append -> kv4_evict

and a token, for all sequences at once, through

    vq_gemv / vq_gemm -> rotary positions -> kv4_append -> kv4_attend -> ... -> kv4_evict

Attention with a budget keeps the newest tokens and those that queries have
looked at most.  Needs an MI355X and the built library.
"""
import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import compressed_index_matmul_amd as vq  # noqa: E402
import vqsynth  # noqa: E402


def synthetic_weight(n_out, k_in, seed):
    sw = vqsynth.random_weight(n_out, k_in, 2, 12, 64, seed=seed)
    return vq.VQWeight(n_out, k_in, 2, 12, 64, codebooks=sw.codebooks, scales=sw.scales, lo=sw.lo, hi=sw.hi)


def rotary(x, pos, base=10000.0):
    """Rotary positions: x [tokens, heads, d] float32, pos int [tokens]."""
    half = x.shape[-1] // 2
    freq = base ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = pos.float()[:, None] * freq
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


class AttentionLayer:
    """Compressed projections around attention; the cache and its lengths."""

    def __init__(self, n_seqs, d_model=576, hq=9, hkv=3, d=64, keep=256, recent=64, max_len=2048, page=64, seed=0):
        self.hq, self.hkv, self.d, self.keep, self.recent = hq, hkv, d, keep, recent
        pages = -(-max_len // page)
        self.capacity = pages * page
        if not 1 <= keep < self.capacity:  # a token is stored before the budget is enforced
            raise ValueError(f"keep={keep} leaves no free slot in a cache of {self.capacity} slots a sequence")
        self.wqkv = synthetic_weight((hq + 2 * hkv) * d, d_model, seed)
        self.wo = synthetic_weight(d_model, hq * d, seed + 1)
        self.cache = vq.KV4Cache(n_seqs * pages, page, hkv, d)
        dev = self.cache.device
        self.table = torch.arange(n_seqs * pages, dtype=torch.int32, device=dev).view(n_seqs, pages)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=dev)      # slots in use, the same for every head
        self.next_pos = torch.zeros(n_seqs, dtype=torch.int32, device=dev)  # tokens seen
        self.step_cu = torch.arange(n_seqs + 1, dtype=torch.int32, device=dev)
        self.max_len = 0  # the host's bound on lens

    def _project(self, w, x):
        return (vq.vq_gemv if x.shape[0] <= 16 else vq.vq_gemm)(w, x)

    def _qkv(self, x, pos):
        y = self._project(self.wqkv, x).view(x.shape[0], -1, self.d)
        q, k, v = y.split([self.hq, self.hkv, self.hkv], 1)
        return rotary(q, pos).to(x.dtype), rotary(k, pos), v

    def _evict(self):
        if self.max_len <= self.keep:
            return
        vq.kv4_evict(self.cache, self.table, self.lens, self.next_pos, keep=self.keep, recent=self.recent,
                     max_len=self.max_len)
        self.lens.clamp_(max=self.keep)
        self.max_len = self.keep

    def prompt(self, x, lengths):
        """x bfloat16 [sum(lengths), d_model]: the packed prompts."""
        if max(lengths) > self.capacity:
            raise ValueError(f"a prompt of {max(lengths)} tokens in a cache of {self.capacity} slots a sequence")
        dev = x.device
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)
        pos = torch.cat([torch.arange(n, device=dev) for n in lengths])
        q, k, v = self._qkv(x, pos)
        kh = k.to(x.dtype)
        out, lse = vq.attn_prompt(q, kh, v.to(x.dtype), cu, return_lse=True)
        got = vq.attn_prompt_weights(q, kh, lse, cu)
        vq.kv4_append(self.cache, k.contiguous(), v, cu, self.table, weights=got)  # float32 rows, as the product gives them
        self.lens += cu[1:] - cu[:-1]
        self.next_pos += cu[1:] - cu[:-1]
        self.max_len = max(lengths)
        self._evict()
        return self._project(self.wo, out.view(x.shape[0], -1))

    def token(self, x):
        """x bfloat16 [sequences, d_model]: the next token of every sequence."""
        q, k, v = self._qkv(x, self.next_pos)
        vq.kv4_append(self.cache, k.contiguous(), v, self.step_cu, self.table, start=self.lens, pos=self.next_pos)
        self.lens += 1
        self.next_pos += 1
        self.max_len += 1
        out = vq.kv4_attend(q, self.cache, self.table, self.lens, max_len=self.max_len, add_weights=True)
        self._evict()
        return self._project(self.wo, out.view(x.shape[0], -1))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--keep", type=int, default=256)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    lengths = [700, 1, 333, 90]
    layer = AttentionLayer(len(lengths), keep=args.keep, recent=min(64, args.keep), seed=args.seed)
    gen = torch.Generator(device="cuda").manual_seed(args.seed)
    x = torch.randn((sum(lengths), 576), generator=gen, device="cuda").bfloat16()
    y = layer.prompt(x, lengths)
    print(f"prompts of {lengths}: output {tuple(y.shape)}, cache lengths {layer.lens.tolist()}")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(args.steps):
        y = layer.token(torch.randn((len(lengths), 576), generator=gen, device="cuda").bfloat16())
    b.record()
    b.synchronize()
    print(f"{args.steps} tokens a sequence: {a.elapsed_time(b) / args.steps * 1e3:.0f} us a step, cache lengths "
          f"{layer.lens.tolist()}, finite {bool(torch.isfinite(y).all())}")


if __name__ == "__main__":
    main()
