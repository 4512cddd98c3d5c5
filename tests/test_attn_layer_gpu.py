"""The example layer end to end: its attention, on the q, k and v its
projections give, against the float64 oracle, through prompt, eviction and
single tokens."""
import importlib.util
import os

import numpy as np
import pytest

import oracle.attention as oa
from attntest import check, host_pool
from vqtest import ROOT, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    ensure_built()
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_layer(example):
    import torch
    vq = example.vq
    lengths = [90, 1, 33]
    layer = example.AttentionLayer(3, keep=48, recent=16, max_len=128, page=32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    seen = {}
    attend, evict, prompt = vq.kv4_attend, vq.kv4_evict, vq.attn_prompt

    def watch_attend(q, cache, table, lens, **kw):
        pool, n = host_pool(cache), lens.tolist()
        out = attend(q, cache, table, lens, **kw)
        d = q.shape[2]
        ref, _, _, mag, vsum, smag = oa.attend_ref(q.double().cpu().numpy(), pool, table.cpu().numpy(), n, d ** -0.5)
        check(out, ref, oa.prompt_bound(ref, mag, vsum, smag.T, d, max(n), "bf16", "fp16", 2.0 ** -11), "token")
        seen["tokens"] = seen.get("tokens", 0) + 1
        return out

    def watch_evict(cache, table, lens, next_pos, keep, recent, max_len):
        pool, n = host_pool(cache), lens.tolist()
        evict(cache, table, lens, next_pos, keep=keep, recent=recent, max_len=max_len)
        pool.evict(table.cpu().numpy(), n, next_pos.tolist(), keep, recent)
        np.testing.assert_array_equal(cache.codes.cpu().numpy(), pool.codes)
        np.testing.assert_array_equal(cache.pos.cpu().numpy(), pool.pos)
        seen["evictions"] = seen.get("evictions", 0) + 1

    def watch_prompt(q, k, v, cu, **kw):
        out, lse = prompt(q, k, v, cu, **kw)
        q64, k64, v64 = (x.double().cpu().numpy() for x in (q, k, v))
        c, d = cu.tolist(), q.shape[2]
        ref, lref, mag, vsum, smag = oa.prompt_ref(q64, k64, v64, c, c, d ** -0.5, True)
        check(out, ref, oa.prompt_bound(ref, mag, vsum, smag, d, max(lengths), "bf16"), "prompt")
        check(lse, lref, oa.lse_bound(lref, smag, d, max(lengths)), "lse")
        return out, lse

    example.vq.kv4_attend, example.vq.kv4_evict, example.vq.attn_prompt = watch_attend, watch_evict, watch_prompt
    try:
        y = layer.prompt(torch.randn((sum(lengths), 576), generator=gen, device="cuda").bfloat16(), lengths)
        assert y.shape == (sum(lengths), 576) and layer.lens.tolist() == [48, 1, 33]
        for _ in range(20):
            y = layer.token(torch.randn((3, 576), generator=gen, device="cuda").bfloat16())
        assert layer.lens.tolist() == [48, 21, 48] and layer.next_pos.tolist() == [110, 21, 53]
        assert bool(torch.isfinite(y).all())
    finally:
        example.vq.kv4_attend, example.vq.kv4_evict, example.vq.attn_prompt = attend, evict, prompt
    assert seen == {"tokens": 20, "evictions": 21}
    # the newest tokens are all there, in every head
    pos = layer.cache.pos[layer.table[0].long()].cpu().numpy().transpose(1, 0, 2).reshape(3, -1)[:, :48]
    for h in range(3):
        assert set(range(110 - 16, 110)) <= set(pos[h].tolist())
