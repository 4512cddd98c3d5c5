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
