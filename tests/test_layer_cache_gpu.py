"""What the example layer's cache is given: the products' float32 rows."""
import numpy as np
import pytest

import oracle.attention as oa
from attntest import check
from test_attn_layer_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,norm", [(None, False), (30, True)])
def test_cached_rows_keep_the_products_bits(example, monkeypatch, window, norm):  # noqa: F811
    """Keys are rotated in float32 and values stored as the product gives them:
    rounding them to 16 bits first would cost the cache a second rounding."""
    import torch
    vq = example.vq
    layer = example.AttentionLayer(2, keep=60, recent=8, max_len=96, page=32, window=window, norm=norm)
    rotate, append, project = vq.attn_rotate, vq.kv4_append, layer._project
    rotated, stored, products = [], [], []

    def watch_project(w, x):
        y = project(w, x)
        if w is layer.wqkv:
            products.append(y.view(x.shape[0], -1, 64))
        return y

    def watch_rotate(q, k, pos, r, **kw):
        rotated.append((k.double().cpu().numpy(), pos.tolist(), kw.get("k_weight")))
        return rotate(q, k, pos, r, **kw)

    def watch_append(cache, k, v, cu, table, **kw):
        stored.append((k.clone(), v.clone()))
        return append(cache, k, v, cu, table, **kw)

    monkeypatch.setattr(layer, "_project", watch_project)
    monkeypatch.setattr(vq, "attn_rotate", watch_rotate)
    monkeypatch.setattr(vq, "kv4_append", watch_append)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rows(n):
        return torch.randn((n, 576), generator=gen, device="cuda").bfloat16()

    layer.prompt(rows(47), [33, 14])
    layer.chunk(rows(7), [5, 2])
    layer.token(rows(2))
    assert len(rotated) == len(stored) == len(products) == 3
    for (k64, pos, w), (k, v), y in zip(rotated, stored, products):
        assert k.dtype == v.dtype == torch.float32
        weight = None if w is None else w.double().cpu().numpy()
        want, mag = oa.rotate_ref(k64, pos, layer.rotary.inv_freq, weight=weight, eps=1e-6)
        check(k, want, oa.rotate_bound(want, mag, 64, "fp32", norm), "keys")
        assert torch.equal(v, y[:, 12:])


def watch_evictions(vq, layer, monkeypatch, seen):
    """Before each eviction: the weights accumulated so far of every sequence's
    slots [heads, slots], their keys, positions and lengths."""
    import torch
    evict = vq.kv4_evict

    def state():
        n = layer.lens.tolist()
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        k, _ = vq.kv4_read(layer.cache, cu, layer.table, max(sum(n), 1), dtype=torch.float32)
        k = k.double().cpu().numpy()

        def of(t):
            return [t[layer.table[b].long()].transpose(0, 1).reshape(t.shape[1], -1)[:, :m].double().cpu().numpy()
                    for b, m in enumerate(n)]

        return dict(n=n, keys=[k[a:b] for a, b in zip(cu.tolist(), cu.tolist()[1:])], weights=of(layer.cache.weights),
                    pos=of(layer.cache.pos))

    def watch(cache, table, lens, next_pos, **kw):
        seen.append(state())
        evict(cache, table, lens, next_pos, **kw)

    monkeypatch.setattr(vq, "kv4_evict", watch)
    return state


@pytest.mark.parametrize("chunks", [[[40, 50, 9]], [[3, 2, 1], [37, 45, 0]], [[0, 0, 30], [0, 20, 0], [41, 0, 0]]])
def test_a_budget_after_chunks_goes_by_what_their_queries_saw(example, monkeypatch, chunks):  # noqa: F811
    """The first eviction after chunks finds in every slot what it had before
    them and the float64 weights of the chunks' queries, and keeps by these."""
    import torch
    vq = example.vq
    keep, recent, d, hq, hkv = 60, 8, 64, 9, 3
    layer = example.AttentionLayer(3, keep=keep, recent=recent, max_len=160, page=32)
    evictions, queries = [], []
    state = watch_evictions(vq, layer, monkeypatch, evictions)
    attend = vq.kv4_attend_chunk

    def watch_attend(q, cache, table, lens, cu=None, **kw):
        queries.append((q.double().cpu().numpy(), cu.tolist(), lens.tolist()))
        return attend(q, cache, table, lens, cu, **kw)

    monkeypatch.setattr(vq, "kv4_attend_chunk", watch_attend)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rows(n):
        return torch.randn((n, 576), generator=gen, device="cuda").bfloat16()

    layer.prompt(rows(101), [50, 40, 11])
    before, made = state(), []
    for lengths in chunks:
        assert all(max(e["n"]) <= keep for e in evictions)  # none that cut a sequence
        first = len(queries)
        layer.chunk(rows(sum(lengths)), lengths)
        made.append(queries[first])
    found, protected = evictions[-1], 0
    assert max(found["n"]) > keep
    for b, n in enumerate(found["n"]):
        want, slack = np.zeros((hkv, n)), np.zeros((hkv, n))
        want[:, :before["n"][b]] = before["weights"][b]
        for q64, cu, lens in made:
            at, keys = [0, cu[b + 1] - cu[b]], found["keys"][b][:lens[b]]
            if at[1] == 0:
                continue
            q = q64[cu[b]:cu[b + 1]]
            _, lse, _, _, _ = oa.prompt_ref(q, keys, keys, at, [0, lens[b]], d ** -0.5, True)
            w, smag = oa.prompt_weights_ref(q, keys, lse, at, [0, lens[b]], d ** -0.5, True, 0)
            want[:, :lens[b]] += w
            # keys are read back in bf16, which moves a score by 2^-8 of its products' sum, and fp16 probabilities and fp32
            # sums are far below that
            slack[:, :lens[b]] += w * np.expm1(smag * (2.0 ** -8 + 2.0 ** -10) * 1.01 + 2.0 ** -10) + 2.0 ** -20
        check(torch.from_numpy(found["weights"][b]), want, slack + 2.0 ** -20 * (1.0 + want), f"weights of sequence {b}")
        # who has to be kept: more weight, whatever the rounding, than all but the budget's part of the other slots
        if n <= keep:
            continue
        kept = layer.cache.pos[layer.table[b].long()].transpose(0, 1).reshape(hkv, -1)[:, :keep].cpu().numpy()
        for h in range(hkv):
            pos, next_pos = found["pos"][b][h], int(layer.next_pos[b])
            old = pos < next_pos - recent
            low, high = (want - slack)[h], (want + slack)[h]
            for i in np.nonzero(old)[0]:
                if (high[old] >= low[i]).sum() <= keep - recent:
                    assert pos[i] in kept[h], (b, h, pos[i])
                    protected += pos[i] >= next_pos - sum(c[b] for c in chunks)
    assert protected > 0  # tokens of the chunks among them, older than the newest
