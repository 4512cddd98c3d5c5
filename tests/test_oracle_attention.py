"""Pins of the attention oracle: values worked out by hand, and identities
that hold for any input."""
import math

import numpy as np
import pytest

import oracle.attention as oa


def test_softmax_rows_by_hand():
    p, lse = oa.softmax_rows(np.array([[0.0, math.log(3.0), -np.inf], [-np.inf] * 3]))
    np.testing.assert_allclose(p, [[0.25, 0.75, 0.0], [0.0, 0.0, 0.0]], atol=1e-15)
    assert abs(lse[0] - math.log(4.0)) < 1e-15 and np.isneginf(lse[1])


def test_prompt_by_hand():
    """Two queries, three keys, one channel in use: causal sees 2 and 3 keys."""
    q, k, v = np.zeros((2, 1, 4)), np.zeros((3, 1, 4)), np.zeros((3, 1, 4))
    q[:, 0, 0] = 1.0
    k[:, 0, 0] = [0.0, math.log(2.0), math.log(5.0)]
    v[:, 0, 1] = [1.0, 4.0, 8.0]
    out, lse, *_ = oa.prompt_ref(q, k, v, [0, 2], [0, 3], 1.0, True)
    np.testing.assert_allclose(out[:, 0, 1], [(1 + 8) / 3, (1 + 8 + 40) / 8], rtol=1e-15)
    np.testing.assert_allclose(lse[0], [math.log(3.0), math.log(8.0)], rtol=1e-15)
    w, _ = oa.prompt_weights_ref(q, k, lse, [0, 2], [0, 3], 1.0, True, 0)
    np.testing.assert_allclose(w[0], [1 / 3 + 1 / 8, 2 / 3 + 2 / 8, 5 / 8], rtol=1e-15)
    w, _ = oa.prompt_weights_ref(q, k, lse, [0, 2], [0, 3], 1.0, True, 1)
    np.testing.assert_allclose(w[0], [1 / 8, 2 / 8, 5 / 8], rtol=1e-15)


def test_prompt_rows_without_keys():
    q, k = np.ones((3, 2, 4)), np.ones((1, 1, 4))
    out, lse, *_ = oa.prompt_ref(q, k, k, [0, 3], [0, 1], 1.0, True)  # queries 0 and 1 see nothing
    assert (out[:2] == 0).all() and np.isneginf(lse[:, :2]).all() and (out[2] == 1).all()


def test_encode_by_hand():
    """0 .. 31 / 2: step fp16(15.5 / 15), codes by rounding."""
    x = (np.arange(32) / 2).astype(np.float32)
    c, s, m = oa.kv4_encode(x)
    step = float(np.float16(15.5 / 15))
    assert m[0] == 0 and float(s[0]) == step
    assert c.tolist() == [round(float(v) / step) for v in x]
    assert np.abs(oa.kv4_values(c, s, m) - x).max() <= step / 2 + 15 * 2.0 ** -10


@pytest.mark.parametrize("x,code,step,low", [
    (np.full(32, 2.5), 0, 0.0, 2.5),                       # a constant group
    (np.full(32, 1e6), 0, 0.0, 32768.0),                   # saturated
    (np.concatenate([np.full(16, -np.inf), np.full(16, np.inf)]), None, 4368.0, -32768.0),  # fp16(65536 / 15)
])
def test_encode_edges(x, code, step, low):
    c, s, m = oa.kv4_encode(x.astype(np.float32))
    assert float(s[0]) == step and float(m[0]) == low
    assert c.tolist() == ([code] * 32 if code is not None else [0] * 16 + [15] * 16)


def test_encode_nan_takes_its_group_only():
    x = np.arange(64, dtype=np.float32)
    x[3] = np.nan
    c, s, m = oa.kv4_encode(x)
    assert np.isnan(m[0]) and np.isnan(s[0]) and (c[:32] == 0).all() and float(m[1]) == 32.0


def empty_pool(pages, heads, page, d):
    return oa.Pool(np.zeros((pages, 2, heads, page * d // 2), np.uint8),
                   np.zeros((pages, 2, heads, page // 4, d // 32, 8), np.float16),
                   np.zeros((pages, heads, page), np.float32), np.zeros((pages, heads, page), np.int32))


def test_layout_by_hand():
    """D = 64 (DG = 2).  Channel 13 is nibble 5 of octet 1: word 1 * 2 + 0, so
    byte 8 + 2, high bits; channel 40 is nibble 0 of octet 5 = 4 + 1: word
    1 * 2 + 1.  A value's channel 40 of slot 6 (third of its four: position 1)
    is byte (40 / 2) * 4 + 1 of the second block of 128, low bits."""
    pool = empty_pool(1, 1, 32, 64)
    c = np.zeros(64, np.uint8)
    c[13], c[40] = 7, 9
    for kind in (0, 1):
        pool.put(kind, 0, 0, 6, c, np.float16([1, 2]), np.float16([3, 4]))
    keys, values = pool.codes[0, 0, 0], pool.codes[0, 1, 0]
    assert keys[6 * 32 + 2 * 4 + 2] == 7 << 4 and keys[6 * 32 + 3 * 4] == 9 and (keys > 0).sum() == 2
    assert values[128 + 20 * 4 + 1] == 9 and values[128 + 6 * 4 + 1] == 7 << 4 and (values > 0).sum() == 2
    assert pool.scales[0, 0, 0, 1].tolist() == [[0, 0, 1, 0, 0, 0, 3, 0], [0, 0, 2, 0, 0, 0, 4, 0]]


@pytest.mark.parametrize("d", [64, 128, 256])
def test_layout_is_one_to_one(d):
    """Every nibble of a page belongs to one slot and channel."""
    rng = np.random.default_rng(d)
    pool = empty_pool(1, 1, 32, d)
    want = rng.integers(0, 16, (2, 32, d)).astype(np.uint8)
    for kind in (0, 1):
        for at in range(32):
            pool.put(kind, 0, 0, at, want[kind, at], np.zeros(d // 32), np.zeros(d // 32))
    for kind in (0, 1):
        for at in range(32):
            assert (pool.get(kind, 0, 0, at)[0] == want[kind, at]).all()


def test_evict_by_hand():
    pool = empty_pool(1, 1, 32, 64)
    pool.weights[0, 0, :8] = [5, 1, np.nan, 3, 3, 0, 3, 2]
    pool.pos[0, 0, :8] = np.arange(8)
    # keep 5: the two newest (6, 7), then 0 (5), 3 and 4 (3 each); 6 and 7 move into 1 and 2
    pool.evict(np.zeros((1, 1), np.int32), [8], [8], 5, 2)
    assert pool.pos[0, 0, :8].tolist() == [0, 6, 7, 3, 4, 5, 6, 7]
    assert pool.weights[0, 0, :5].tolist() == [5, 3, 2, 3, 3]
