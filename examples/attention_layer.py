"""The attention half of one decoder layer on compressed weights: prompts,
then single tokens, over a 4-bit cache that is kept to a budget, or under a
sliding window.

    python examples/attention_layer.py [--steps N] [--keep N] [--window N] [--sinks N] [--chunk N] [--seed N]

The q/k/v and output projections are 2-stage 12-bit codebook weights
(SmolLM-135M's shape: rows of 576, 9 query and 3 key/value heads of 64); all
weights and inputs are synthetic.  A prompt goes through

    vq_gemm -> attn_rotate -> attn_prompt -> vq_gemm
                           -> attn_prompt_weights -> kv4_append -> kv4_evict

and a token, for all sequences at once, through

    vq_gemv / vq_gemm -> attn_rotate -> kv4_append -> kv4_attend -> ... -> kv4_evict

Attention with a budget keeps the newest tokens and those that queries have
looked at most.  With a window every token sees the newest ones and the first
few, and nothing is evicted:

    attn_rotate -> attn_prompt (window) -> ...       kv4_append -> kv4_attend_chunk (window) -> ...

Several tokens a sequence at once (the next piece of a prompt, drafted tokens)
go through kv4_append and kv4_attend_chunk in either case.  Under a budget what
their queries looked at is counted when slots have to go:

    kv4_attend_chunk (log sums) -> kv4_read -> attn_prompt_weights -> kv4_evict

Needs an MI355X and the built library.
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


class AttentionLayer:
    """Compressed projections around attention; the cache and its lengths."""

    def __init__(self, n_seqs, d_model=576, hq=9, hkv=3, d=64, keep=256, recent=64, max_len=2048, page=64, seed=0,
                 window=None, sinks=0, norm=False):
        self.hq, self.hkv, self.d, self.keep, self.recent = hq, hkv, d, keep, recent
        self.window, self.sinks = window, sinks
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
        self.chunks = []  # since the last eviction: queries, their offsets, the lengths after them, bounds on both
        self.rotary = vq.Rotary(d, device=dev)
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.norms = [1.0 + 0.1 * torch.randn(d, generator=gen, device=dev) for _ in range(2)] if norm else [None, None]

    def _project(self, w, x):
        return (vq.vq_gemv if x.shape[0] <= 16 else vq.vq_gemm)(w, x)

    def _qkv(self, x, pos):
        y = self._project(self.wqkv, x).view(x.shape[0], -1, self.d)
        q, k, v = y.split([self.hq, self.hkv, self.hkv], 1)
        q, k = vq.attn_rotate(q, k, pos, self.rotary, q_weight=self.norms[0], k_weight=self.norms[1])
        return q.to(x.dtype), k, v  # the cache takes float32 rows, as the product gives them

    def _evict(self):
        if self.window is not None or self.max_len <= self.keep:
            return
        for chunk in self.chunks:
            self._count(*chunk)
        self.chunks.clear()
        vq.kv4_evict(self.cache, self.table, self.lens, self.next_pos, keep=self.keep, recent=self.recent,
                     max_len=self.max_len)
        self.lens.clamp_(max=self.keep)
        self.max_len = self.keep

    def _count(self, q, cu, lens, max_q, max_len):
        """Adds what a chunk's queries gave each slot to the cache's weights.  Only evictions need it, so it waits for
        one: no slot moves before.  Keys are read back in q's 16 bits, which a ranking can bear."""
        _, lse = vq.kv4_attend_chunk(q, self.cache, self.table, lens, cu, max_len=max_len, max_q=max_q, return_lse=True)
        n, ps = len(lens), self.cache.page_size
        ends = lens.cumsum(0, dtype=torch.int32)
        rows = torch.arange(n * max_len, dtype=torch.int32, device=q.device)  # more than there are: lens is not on the host
        cu_k = torch.cat([ends.new_zeros(1), ends])
        k, _ = vq.kv4_read(self.cache, cu_k, self.table, len(rows), dtype=q.dtype)
        got = torch.zeros((self.hkv, len(rows)), device=q.device)
        vq.attn_prompt_weights(q, k, lse, cu, cu_k, out=got)  # rows of no sequence keep their zeros
        seq = torch.searchsorted(ends, rows, right=True).clamp_(max=n - 1)
        slot = (rows - cu_k[seq]).clamp_(max=self.capacity - 1)
        page = self.table[seq, slot // ps].long()
        heads = torch.arange(self.hkv, device=q.device)
        self.cache.weights.index_put_((page[:, None], heads, (slot % ps).long()[:, None]), got.T, accumulate=True)

    def prompt(self, x, lengths):
        """x bfloat16 [sum(lengths), d_model]: the packed prompts."""
        if max(lengths) > self.capacity:
            raise ValueError(f"a prompt of {max(lengths)} tokens in a cache of {self.capacity} slots a sequence")
        dev = x.device
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)
        pos = torch.cat([torch.arange(n, dtype=torch.int32, device=dev) for n in lengths])
        q, k, v = self._qkv(x, pos)
        kh, vh = k.to(x.dtype), v.to(x.dtype)
        if self.window is None:
            out, lse = vq.attn_prompt(q, kh, vh, cu, return_lse=True)
            got = vq.attn_prompt_weights(q, kh, lse, cu)
        else:
            out, got = vq.attn_prompt(q, kh, vh, cu, window=self.window, sinks=self.sinks), None
        vq.kv4_append(self.cache, k, v, cu, self.table, weights=got)
        self.lens += cu[1:] - cu[:-1]
        self.next_pos += cu[1:] - cu[:-1]
        self.max_len = max(lengths)
        self._evict()
        return self._project(self.wo, out.view(x.shape[0], -1))

    def chunk(self, x, lengths):
        """x bfloat16 [sum(lengths), d_model]: the next lengths[b] tokens of every
        sequence, packed."""
        if self.max_len + max(lengths) > self.capacity:
            raise ValueError(f"{max(lengths)} tokens after {self.max_len} in a cache of {self.capacity} slots a sequence")
        dev = x.device
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)
        n = cu[1:] - cu[:-1]
        seq = torch.repeat_interleave(torch.arange(len(lengths), device=dev), n, output_size=sum(lengths))
        pos = torch.arange(sum(lengths), dtype=torch.int32, device=dev) + (self.next_pos - cu[:-1])[seq]
        q, k, v = self._qkv(x, pos)
        vq.kv4_append(self.cache, k, v, cu, self.table, start=self.lens, pos=self.next_pos)
        self.lens += n
        self.next_pos += n
        self.max_len += max(lengths)
        out = vq.kv4_attend_chunk(q, self.cache, self.table, self.lens, cu, window=self.window, sinks=self.sinks,
                                  max_len=self.max_len, max_q=max(lengths))
        if self.window is None:
            self.chunks.append((q, cu, self.lens.clone(), max(lengths), self.max_len))
        self._evict()
        return self._project(self.wo, out.view(x.shape[0], -1))

    def token(self, x):
        """x bfloat16 [sequences, d_model]: the next token of every sequence."""
        if self.max_len >= self.capacity:
            raise ValueError(f"a token after {self.max_len} in a cache of {self.capacity} slots a sequence")
        q, k, v = self._qkv(x, self.next_pos)
        vq.kv4_append(self.cache, k, v, self.step_cu, self.table, start=self.lens, pos=self.next_pos)
        self.lens += 1
        self.next_pos += 1
        self.max_len += 1
        if self.window is None:
            out = vq.kv4_attend(q, self.cache, self.table, self.lens, max_len=self.max_len, add_weights=True)
        else:
            out = vq.kv4_attend_chunk(q, self.cache, self.table, self.lens, window=self.window, sinks=self.sinks,
                                      max_len=self.max_len)
        self._evict()
        return self._project(self.wo, out.view(x.shape[0], -1))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--keep", type=int, default=256)
    ap.add_argument("--window", type=int, default=None)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--chunk", type=int, default=0, help="tokens a sequence in one further piece of the prompts")
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    lengths = [700, 1, 333, 90]
    layer = AttentionLayer(len(lengths), keep=args.keep, recent=min(64, args.keep), seed=args.seed,
                           window=args.window, sinks=args.sinks)
    gen = torch.Generator(device="cuda").manual_seed(args.seed)
    x = torch.randn((sum(lengths), 576), generator=gen, device="cuda").bfloat16()
    y = layer.prompt(x, lengths)
    print(f"prompts of {lengths}: output {tuple(y.shape)}, cache lengths {layer.lens.tolist()}")
    if args.chunk:
        y = layer.chunk(torch.randn((len(lengths) * args.chunk, 576), generator=gen, device="cuda").bfloat16(),
                        [args.chunk] * len(lengths))
        print(f"{args.chunk} more tokens each: output {tuple(y.shape)}, cache lengths {layer.lens.tolist()}")
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
