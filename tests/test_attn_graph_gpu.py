"""Prompt attention, gathered weights and the cache read in captured graphs,
in one launch and in pieces that meet in a second: every replay equals the
eager call on the same inputs, bit for bit, with eager work between replays."""
import numpy as np
import pytest

from attntest import heads, ints, new_cache, offsets
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (4, 4, 128), (2, 1, 256)])
@pytest.mark.parametrize("lens,klens", [([40, 1, 700], [40, 1, 700]), ([30, 0, 9], [2600, 20, 600])])
def test_prompt_weights_and_read(vq, lens, klens, hq, hkv, d, kind):
    import torch
    rng = np.random.default_rng(d)
    _, cu = offsets(lens)
    _, ck = offsets(klens)
    total = sum(klens)
    q, _ = heads(rng, sum(lens), hq, d, kind)
    k, _ = heads(rng, total, hkv, d, kind)
    per = max(klens) // 64 + 1
    cache = new_cache(vq, per * len(lens), 64, hkv, d)
    table = torch.arange(per * len(lens), dtype=torch.int32, device="cuda").view(len(lens), per)
    out = torch.empty_like(q)
    w = torch.empty((hkv, total), device="cuda")

    def step():
        vq.kv4_append(cache, k, k, ck, table)
        rk, rv = vq.kv4_read(cache, ck, table, total, dtype=k.dtype)
        _, lse = vq.attn_prompt(q, rk, rv, cu, ck, out=out, return_lse=True)
        vq.attn_prompt_weights(q, rk, lse, cu, ck, out=w)
        return rk, rv, lse

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for i in range(4):
        q.copy_(torch.randn_like(q, dtype=torch.float32).to(q.dtype))
        k.copy_(torch.randn_like(k, dtype=torch.float32).to(k.dtype))
        eager = [t.clone() for t in (*step(), out, w)]
        for t in (*held, out, w):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip((*held, out, w), eager)):
            assert torch.equal(a, b), (i, j)
