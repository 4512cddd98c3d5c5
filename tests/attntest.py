"""Helpers of the attention tests: random packed heads, caches, and checks
against the oracle's bounds."""
from __future__ import annotations

import numpy as np

import oracle.attention as oa


def torch_type(kind):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[kind]


def heads(rng, n, h, d, kind, scale=1.0, offset=0.0):
    """Random [n, h, d] of the type on the GPU, and its float64 values."""
    import torch
    x = torch.from_numpy((rng.standard_normal((n, h, d)) * scale + offset * rng.standard_normal((1, h, d)))
                         .astype(np.float32)).to(torch_type(kind))
    return x.cuda(), x.double().numpy()


def offsets(lens):
    import torch
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def ints(values):
    import torch
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def check(got, want, bound, what):
    """|got - want| within the bound, infinities and NaN in the same places."""
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(got)), f"{what}: non-finite values differ"
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True), f"{what}: non-finite values differ"
    err = np.abs(np.where(fin, got, 0.0) - np.where(fin, want, 0.0))
    bad = err > np.broadcast_to(bound, err.shape)
    i = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else ()
    assert not bad.any(), f"{what}: {bad.sum()} outside, worst at {i}: {got[i]} for {want[i]}"


def new_cache(vq, pages, page, heads_, d, fill=0xFF):
    """A cache whose unwritten bytes are all `fill` (0xFF: NaN steps)."""
    cache = vq.KV4Cache(pages, page, heads_, d)
    cache.codes.fill_(fill)
    cache.scales.view(dtype=cache.pos.dtype).fill_(-1 if fill == 0xFF else 0)
    cache.weights.fill_(float("nan"))
    cache.pos.fill_(-7)
    return cache


def host_pool(cache):
    return oa.Pool(cache.codes.cpu().numpy(), cache.scales.cpu().numpy(), cache.weights.cpu().numpy(),
                   cache.pos.cpu().numpy())


def same_pool(cache, pool, what):
    np.testing.assert_array_equal(cache.codes.cpu().numpy(), pool.codes, err_msg=what)
    np.testing.assert_array_equal(cache.scales.cpu().numpy().view(np.uint16), pool.scales.view(np.uint16), err_msg=what)
    np.testing.assert_array_equal(cache.weights.cpu().numpy(), pool.weights, err_msg=what)
    np.testing.assert_array_equal(cache.pos.cpu().numpy(), pool.pos, err_msg=what)


def block_table(rng, n, per, pages):
    return rng.permutation(pages)[:n * per].reshape(n, per).astype(np.int32)
