"""The 4-bit cache: append and read back bit for bit against the oracle,
single-token attention within the bounds derived from its roundings, eviction
exactly."""
import numpy as np
import pytest

import oracle.attention as oa
from attntest import block_table, check, heads, host_pool, ints, new_cache, offsets, same_pool, torch_type
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hkv,d,page", [(3, 64, 32), (2, 128, 64), (1, 256, 96)])
def test_append_and_read(vq, hkv, d, page, kind):
    """Ragged rows at every alignment within a quad, over page ends; the pool
    equals the oracle's byte for byte, so untouched slots keep theirs."""
    import torch
    rng = np.random.default_rng(d)
    lens, start = [1, 2, 3, 4, 5, 0, 37, 130, 6, 1, 4], [0, 1, 2, 3, 30, 7, 31, 5, page - 2, page - 1, 4]
    per = 1 + max(a + b for a, b in zip(lens, start)) // page
    table = block_table(rng, len(lens), per, len(lens) * per + 2)
    cache = new_cache(vq, table.size + 2, page, hkv, d)
    pool = host_pool(cache)
    cu, cu_d = offsets(lens)
    k, k64 = heads(rng, cu[-1], hkv, d, kind, 1.0, 3.0)
    v, v64 = heads(rng, cu[-1], hkv, d, kind, 0.01)
    t, s = torch.from_numpy(table).cuda(), ints(start)
    vq.kv4_append(cache, k, v, cu_d, t, s)
    pool.append(k64.astype(np.float32), v64.astype(np.float32), cu, table, start)
    same_pool(cache, pool, "append")
    # a second chunk after the first, with positions and weights given
    start2 = [a + b for a, b in zip(start, lens)]
    lens2 = [3] * len(lens)
    cu2, cu2_d = offsets(lens2)
    fits = [min(n, per * page) for n in start2]
    k2, k264 = heads(rng, cu2[-1], hkv, d, kind)
    w2 = rng.random((hkv, cu2[-1])).astype(np.float32)
    p2 = [100 * i for i in range(len(lens))]
    vq.kv4_append(cache, k2, k2, cu2_d, t, ints(fits), pos=ints(p2), weights=torch.from_numpy(w2).cuda())
    pool.append(k264.astype(np.float32), k264.astype(np.float32), cu2, table, fits, p2, w2)
    same_pool(cache, pool, "second append")
    # read the first rows back
    for out in ("fp32", "bf16", "fp16"):
        rk, rv = vq.kv4_read(cache, cu_d, t, int(cu[-1]), start=s, dtype=torch_type(out))
        for got, kd in ((rk, 0), (rv, 1)):
            want = np.zeros((cu[-1], hkv, d))
            for b in range(len(lens)):
                for h in range(hkv):
                    for i in range(lens[b]):
                        slot = start[b] + i
                        want[cu[b] + i, h] = oa.kv4_values(*pool.get(kd, h, table[b, slot // page], slot % page))
            want = torch.from_numpy(want).float().to(torch_type(out))  # each value is fp32, then rounded once
            assert torch.equal(got.cpu(), want), (out, kd)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_append_edge_values(vq, kind):
    """Constant groups, zeros of both signs, tiny and huge values, infinities,
    NaN, one outlier: codes, steps and minima equal the oracle's."""
    import torch
    rows = [np.zeros(64), np.full(64, -0.0), np.full(64, 2.5), np.full(64, 1e-30), np.linspace(-1e-6, 1e-6, 64),
            np.linspace(-6e4, 6e4, 64), np.full(64, np.inf), np.linspace(-1, 1, 64), np.linspace(-1, 1, 64),
            np.concatenate([[4e4], np.full(63, 1e-3)]), np.full(64, -3e38), np.linspace(1000, 1001, 64)]
    rows[7][5] = np.nan
    rows[8][40] = -np.inf
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(torch_type(kind)).view(len(rows), 1, 64)
    cache = new_cache(vq, 1, 32, 1, 64)
    pool = host_pool(cache)
    cu, cu_d = offsets([len(rows)])
    vq.kv4_append(cache, x.cuda(), x.cuda(), cu_d, ints([[0]]), ints([1]))
    f = x.float().numpy()
    pool.append(f, f, cu, np.zeros((1, 1), np.int32), [1])
    got, want = cache.scales.cpu().numpy(), pool.scales
    np.testing.assert_array_equal(cache.codes.cpu().numpy(), pool.codes)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_append_past_the_table(vq):
    """Rows past the block table's capacity are dropped, read back as zeros."""
    import torch
    rng = np.random.default_rng(2)
    cache = new_cache(vq, 3, 32, 2, 64)
    pool = host_pool(cache)
    cu, cu_d = offsets([40, 3])
    k, k64 = heads(rng, 43, 2, 64, "bf16")
    table = np.array([[1], [0]], np.int32)
    t = torch.from_numpy(table).cuda()
    vq.kv4_append(cache, k, k, cu_d, t, ints([5, 2000]))
    pool.append(k64.astype(np.float32), k64.astype(np.float32), cu, table, [5, 2000])
    same_pool(cache, pool, "append")
    rk, rv = vq.kv4_read(cache, cu_d, t, 43, start=ints([5, 2000]))
    assert bool((rk[27:] == 0).all()) and bool((rv[27:] == 0).all()) and bool((rk[:27] != 0).any())


def test_append_strided_and_stream(vq):
    """Slices of a fused row and head-major rows, on another stream."""
    import torch
    rng = np.random.default_rng(3)
    _, cu_d = offsets([30, 11])
    t = ints([[0], [1]])
    k, _ = heads(rng, 41, 2, 128, "bf16")
    v, _ = heads(rng, 41, 2, 128, "bf16")
    a = new_cache(vq, 2, 32, 2, 128)
    vq.kv4_append(a, k, v, cu_d, t)
    fused = torch.cat([k, v], 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, c = new_cache(vq, 2, 32, 2, 128), new_cache(vq, 2, 32, 2, 128)
    side.wait_stream(torch.cuda.current_stream())
    vq.kv4_append(b, fused[:, :2], fused[:, 2:], cu_d, t, stream=side)
    vq.kv4_append(c, k.transpose(0, 1).contiguous().transpose(0, 1), v.transpose(0, 1).contiguous().transpose(0, 1), cu_d, t,
                  stream=side.cuda_stream)
    ka, va = vq.kv4_read(a, cu_d, t, 41)
    kb, vb = vq.kv4_read(b, cu_d, t, 41, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.codes, c.codes)
    assert torch.equal(a.scales.view(torch.int16), b.scales.view(torch.int16))
    assert torch.equal(ka, kb) and torch.equal(va, vb)


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
def filled(vq, rng, lens, hkv, d, page, spare=2, offset=1.5):
    """A cache whose first lens[b] slots hold random tokens, all else NaN."""
    import torch
    per = max(1, -(-max(lens) // page))
    table = block_table(rng, len(lens), per, len(lens) * per + spare)
    cache = new_cache(vq, table.size + spare, page, hkv, d)
    cu, cu_d = offsets(lens)
    k, _ = heads(rng, cu[-1], hkv, d, "fp32", 1.0, offset)
    v, _ = heads(rng, cu[-1], hkv, d, "fp32")
    t = torch.from_numpy(table).cuda()
    w = torch.from_numpy(rng.random((hkv, cu[-1])).astype(np.float32)).cuda()
    vq.kv4_append(cache, k, v, cu_d, t, weights=w)
    return cache, table, t


def attend(vq, kind, hq, hkv, d, page, lens, scale=None, seed=0, spread=1.0, max_len=None, caps=None):
    rng = np.random.default_rng(seed)
    scale = d ** -0.5 if scale is None else scale
    cache, table, t = filled(vq, rng, lens, hkv, d, page)
    q, q64 = heads(rng, len(lens), hq, d, kind, spread)
    before = host_pool(cache)
    weights0 = cache.weights.clone()
    counted = lens if caps is None else [min(n, caps) for n in lens]
    ref, lref, probs, mag, vsum, smag = oa.attend_ref(q64, before, table, counted, scale)
    n = max([1, *counted])
    bound = oa.prompt_bound(ref, mag, vsum, smag.T, d, n, kind, p_kind="fp16", v_round=2.0 ** -11)
    out, lse = vq.kv4_attend(q, cache, t, ints(lens), scale=scale, max_len=max_len, return_lse=True)
    check(out, ref, bound, "out")
    check(lse, lref, oa.lse_bound(lref, smag, d, n), "lse")
    np.testing.assert_array_equal(cache.weights.cpu().numpy(), before.weights)
    out2, lse2 = vq.kv4_attend(q, cache, t, ints(lens), scale=scale, max_len=max_len, add_weights=True, return_lse=True)
    check(out2, ref, bound, "out with weights")
    check(lse2, lref, oa.lse_bound(lref, smag, d, n), "lse with weights")
    # the added weights: relative error of a probability, then the fp32 additions
    want, slack = before.weights.astype(np.float64), np.zeros_like(before.weights, dtype=np.float64)
    group = hq // hkv
    rel = 2.0 * (smag * ((d + 8) * 2.0 ** -24 + 2.0 ** -22) + (n + 8) * 2.0 ** -24) + 2.0 ** -20
    for b, c in enumerate(counted):
        slots = np.arange(c)
        pages, at = table[b, slots // page], slots % page
        for h in range(hkv):
            p = probs[b][h * group:(h + 1) * group]
            want[pages, h, at] += p.sum(0)
            slack[pages, h, at] = (p * rel[b, h * group:(h + 1) * group, None]).sum(0) + 2.0 ** -22 * want[pages, h, at]
    check(cache.weights, want, slack + 2.0 ** -40, "weights")
    return cache, t, q, out, weights0


LENS = [1, 2, 3, 5, 31, 32, 33, 64, 100, 127, 128, 129, 300, 0]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d,page", [(3, 1, 64, 32), (4, 2, 128, 64), (2, 1, 256, 96)])
def test_attend_lengths(vq, hq, hkv, d, page, kind):
    attend(vq, kind, hq, hkv, d, page, LENS, seed=d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (9, 3), (16, 1), (17, 1), (20, 2), (35, 1)])
def test_attend_head_groups(vq, hq, hkv):
    attend(vq, "bf16", hq, hkv, 64, 32, [77, 1, 40], seed=hq)


@pytest.mark.parametrize("n", [700, 2500])
def test_attend_splits(vq, n):
    """One sequence cut into many pieces, with short ones beside it."""
    attend(vq, "bf16", 4, 1, 128, 128, [n], seed=n)
    attend(vq, "fp16", 4, 1, 64, 64, [n, 3, 0, 129], seed=n + 1)


@pytest.mark.parametrize("hq,hkv", [(2, 1), (6, 3), (20, 1)])
def test_attend_many_sequences(vq, hq, hkv):
    """More sequences than a wave has lanes, empty ones among them, longer than
    one workgroup takes whole."""
    rng = np.random.default_rng(hq)
    lens = [int(n) for n in rng.integers(0, 90, 150)]
    for i in (0, 63, 64, 65, 127, 128, 149):
        lens[i] = 0
    lens[70] = 1100
    attend(vq, "bf16", hq, hkv, 64, 32, lens, seed=hq)


def test_attend_many_long_rows(vq):
    """More rows than shares and rows longer than one: whole rows, rows cut
    once and rows cut often in the same call."""
    attend(vq, "fp16", 2, 1, 64, 128, [1500, 40, 1200, 0, 64, 2000], seed=21)
    attend(vq, "bf16", 8, 8, 128, 64, [1300, 33], seed=22)


def test_attend_max_len(vq):
    """Lengths beyond max_len count as max_len."""
    attend(vq, "bf16", 4, 2, 64, 32, [300, 10, 200], seed=4, max_len=190, caps=190)
    attend(vq, "bf16", 4, 2, 64, 32, [300, 10, 200], seed=5, max_len=1, caps=1)


def test_attend_large_scores_and_queries(vq):
    attend(vq, "bf16", 4, 2, 128, 32, [150, 40], seed=6, spread=30.0, scale=0.5)
    attend(vq, "bf16", 4, 2, 128, 32, [150, 40], seed=7, spread=1e30, scale=1e-30)   # beyond fp16's range
    attend(vq, "bf16", 4, 2, 128, 32, [150, 40], seed=8, spread=1e-20, scale=1.0)    # below it
    attend(vq, "fp16", 4, 2, 64, 32, [90], seed=9, spread=1e-4, scale=1.0)


def test_attend_all_empty_and_no_sequences(vq):
    import torch
    cache = new_cache(vq, 4, 32, 2, 64)
    q = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    t = ints([[0], [1], [2]])
    for weigh in (False, True):
        for max_len in (None, 0):
            out, lse = vq.kv4_attend(q, cache, t, ints([0, 0, -3]), max_len=max_len, add_weights=weigh, return_lse=True)
            assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    out = vq.kv4_attend(q[:0], cache, t[:0], ints([])[:0])
    assert out.shape == (0, 4, 64)


def test_attend_nan_slot_and_inf_query(vq):
    """A NaN in a slot that counts reaches that sequence and head, no other."""
    import torch
    rng = np.random.default_rng(10)
    cache, table, t = filled(vq, rng, [60, 60], 2, 64, 32)
    q, _ = heads(rng, 2, 4, 64, "bf16")
    want = vq.kv4_attend(q, cache, t, ints([60, 60]))
    cache.scales[int(table[0, 1]), 1, 0, 2, 0, 5] = float("nan")  # value minimum of slot 32 + 9, head 0, sequence 0
    got = vq.kv4_attend(q, cache, t, ints([60, 60]))
    assert bool(torch.isnan(got[0, :2, :32]).all()) and torch.equal(got[0, :2, 32:], want[0, :2, 32:])
    assert torch.equal(got[0, 2:], want[0, 2:]) and torch.equal(got[1], want[1])
    short = vq.kv4_attend(q, cache, t, ints([41, 60]))  # slots 0 .. 40: not that one
    assert bool(torch.isfinite(short).all())


def test_attend_shared_pages_and_table_slack(vq):
    """Two sequences over the same pages, and a table whose unused entries are
    out of range."""
    import torch
    rng = np.random.default_rng(11)
    cache, table, t = filled(vq, rng, [90], 2, 64, 32)
    q, _ = heads(rng, 1, 4, 64, "bf16")
    want = vq.kv4_attend(q, cache, t, ints([90]))
    wide = torch.full((2, 6), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, :t.shape[1]] = t
    wide[:, -1] = -9
    got = vq.kv4_attend(q.expand(2, -1, -1).contiguous(), cache, wide, ints([90, 90]), max_len=96)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[0])


def test_attend_strided_queries_workspace_stream(vq):
    import torch
    rng = np.random.default_rng(12)
    lens = [500, 20, 333]
    cache, table, t = filled(vq, rng, lens, 2, 128, 64)
    q, _ = heads(rng, 3, 8, 128, "bf16")
    want, lse = vq.kv4_attend(q, cache, t, ints(lens), return_lse=True)
    wide = torch.full((3, 12, 128), float("nan"), dtype=q.dtype, device="cuda")
    wide[:, :8] = q
    ws = torch.full((vq.kv4_attend_workspace_size(cache, 3, 8, 512, False) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    got, l2 = vq.kv4_attend(wide[:, :8], cache, t, ints(lens), max_len=512, workspace=ws, out=out, return_lse=True, stream=side)
    side.synchronize()
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want) and torch.equal(l2, lse)


def test_attend_workspace(vq):
    """A workspace of the asked size serves, whatever it holds; a smaller one
    is refused; one for a longer bound does too."""
    import torch
    rng = np.random.default_rng(16)
    lens = [3000, 20, 333]
    cache, table, t = filled(vq, rng, lens, 2, 128, 64)
    q, _ = heads(rng, 3, 8, 128, "bf16")
    for weigh in (False, True):
        need = vq.kv4_attend_workspace_size(cache, 3, 8, 3000, weigh)
        assert need > 0
        cache.weights.zero_()
        want, lse = vq.kv4_attend(q, cache, t, ints(lens), max_len=3000, add_weights=weigh, return_lse=True)
        w = cache.weights.clone()
        cache.weights.zero_()
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        got, l2 = vq.kv4_attend(q, cache, t, ints(lens), max_len=3000, add_weights=weigh, workspace=ws, return_lse=True)
        assert torch.equal(got, want) and torch.equal(l2, lse) and torch.equal(cache.weights, w)
        with pytest.raises(vq.VQError) as e:
            vq.kv4_attend(q, cache, t, ints(lens), max_len=3000, add_weights=weigh, workspace=ws[:need - 16])
        assert e.value.status == -8


def test_attend_graph_replays(vq):
    """Append, attend and evict in a captured graph: every replay equals the
    eager calls, with eager work between the replays."""
    import torch
    rng = np.random.default_rng(13)
    lens = [300, 120]
    cache, table, t = filled(vq, rng, lens, 2, 64, 32)
    twin = vq.KV4Cache.from_buffers(cache.codes.clone(), cache.scales.clone(), cache.weights.clone(), cache.pos.clone())
    cu = ints([0, 1, 2])
    start, after, pos, nxt = ints([200, 100]), ints([201, 101]), ints([500, 400]), ints([501, 401])
    k, _ = heads(rng, 2, 2, 64, "bf16")
    v, _ = heads(rng, 2, 2, 64, "bf16")
    q, _ = heads(rng, 2, 4, 64, "bf16")
    ws = torch.empty(vq.kv4_attend_workspace_size(cache, 2, 4, 320, True), dtype=torch.uint8, device="cuda")
    we = torch.empty(vq.kv4_evict_workspace_size(cache, 2, 64, 320), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step(c, o, w1, w2):
        vq.kv4_append(c, k, v, cu, t, start, pos=pos)
        vq.kv4_attend(q, c, t, after, max_len=320, add_weights=True, out=o, workspace=w1)
        vq.kv4_evict(c, t, after, nxt, keep=64, recent=10, max_len=320, workspace=w2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(cache, out, ws, we)
    torch.cuda.synchronize()
    for i in range(4):
        q.copy_(torch.randn_like(q, dtype=torch.float32).to(q.dtype))
        k.copy_(torch.randn_like(k, dtype=torch.float32).to(k.dtype))
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(q)
        step(twin, eager, None, None)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
        assert torch.equal(cache.codes, twin.codes) and torch.equal(cache.pos, twin.pos), i
        assert torch.equal(cache.weights.view(torch.int32), twin.weights.view(torch.int32)), i


def test_large_pool(vq):
    """Pages beyond 4 GiB of codes, scales' and weights' offsets beyond 2^31
    elements."""
    import torch
    hkv, d, page = 8, 128, 1024
    per_page = 2 * hkv * page * d // 2
    pages = (5 << 30) // per_page
    codes = torch.empty((pages, 2, hkv, page * d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, 2, hkv, page // 4, d // 32, 8), dtype=torch.float16, device="cuda")
    weights = torch.zeros((pages, hkv, page), dtype=torch.float32, device="cuda")
    pos = torch.zeros((pages, hkv, page), dtype=torch.int32, device="cuda")
    big = vq.KV4Cache.from_buffers(codes, scales, weights, pos)
    rng = np.random.default_rng(14)
    n = 1500
    _, cu = offsets([n])
    k, _ = heads(rng, n, hkv, d, "bf16")
    v, _ = heads(rng, n, hkv, d, "bf16")
    q, _ = heads(rng, 1, 16, d, "bf16")
    small = new_cache(vq, 2, page, hkv, d)
    results = []
    for cache, t in ((big, ints([[pages - 1, pages - 2]])), (small, ints([[1, 0]]))):
        vq.kv4_append(cache, k, v, cu, t)
        out = vq.kv4_attend(q, cache, t, ints([n]), add_weights=True)
        vq.kv4_evict(cache, t, ints([n]), ints([n]), keep=700, recent=50)
        results.append((out, vq.kv4_attend(q, cache, t, ints([700])), *vq.kv4_read(cache, ints([0, 700]), t, 700)))
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def evict(vq, hkv, d, page, lens, keep, recent, make, seed=0, shuffle=True, max_len=None):
    import torch
    rng = np.random.default_rng(seed)
    cache, table, t = filled(vq, rng, lens, hkv, d, page)
    w, pos = cache.weights.cpu().numpy(), cache.pos.cpu().numpy()
    nxt = []
    for b, n in enumerate(lens):
        slots = np.arange(n)
        for h in range(hkv):
            w[table[b, slots // page], h, slots % page] = make(rng, n)
            p = np.sort(rng.choice(5 * n + 1, n, replace=False)) if n else slots
            if n:
                p[-1] = 5 * n  # the newest token is everyone's
            pos[table[b, slots // page], h, slots % page] = rng.permutation(p) if shuffle else p
        nxt.append(5 * n + 1)
    cache.weights.copy_(torch.from_numpy(w))
    cache.pos.copy_(torch.from_numpy(pos))
    pool = host_pool(cache)
    counted = lens if max_len is None else [min(n, max_len) for n in lens]
    vq.kv4_evict(cache, t, ints(lens), ints(nxt), keep=keep, recent=recent, max_len=max_len)
    pool.evict(table, counted, nxt, keep, recent)
    same_pool(cache, pool, "evict")


RANDOM = lambda rng, n: rng.random(n).astype(np.float32) ** 4  # noqa: E731


@pytest.mark.parametrize("hkv,d,page", [(3, 64, 32), (2, 128, 64), (1, 256, 96)])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (33, 0), (64, 64), (100, 20)])
def test_evict(vq, hkv, d, page, keep, recent):
    evict(vq, hkv, d, page, [0, 1, keep - 1, keep, keep + 1, 150, 257], keep, recent, RANDOM, seed=keep)


@pytest.mark.parametrize("make", [
    lambda rng, n: np.zeros(n, np.float32),                                   # all equal
    lambda rng, n: rng.integers(0, 3, n).astype(np.float32),                  # many ties
    lambda rng, n: np.where(rng.random(n) < 0.5, -0.0, 0.0).astype(np.float32),  # zeros of both signs are equal
    lambda rng, n: rng.choice(np.float32([np.nan, -np.inf, np.inf, -1, 0, 1e-45, 1]), n),
    lambda rng, n: rng.standard_normal(n).astype(np.float32),                 # both signs
    lambda rng, n: (1 + rng.integers(0, 300, n) * 2.0 ** -23).astype(np.float32),  # differ in the last byte only
], ids=["equal", "ties", "zeros", "special", "signed", "close"])
def test_evict_weights(vq, make):
    evict(vq, 2, 64, 32, [200, 65, 1000], 64, 7, make, seed=1)
    evict(vq, 1, 64, 32, [200, 65, 1000], 64, 64, make, seed=2, shuffle=False)


def test_evict_long(vq):
    """Thousands of slots, and a length that is no multiple of anything."""
    evict(vq, 1, 64, 256, [40001, 3], 5000, 100, RANDOM, seed=3)


@pytest.mark.parametrize("n,keep", [(2048, 2040), (2049, 2040), (5000, 700), (5000, 4990), (16384, 100), (16385, 4000),
                                    (32768, 32760), (32769, 32750), (33000, 9000)])
def test_evict_sizes(vq, n, keep):
    """Both sides of the lengths at which the search changes its form, with
    few and with many slots to move."""
    evict(vq, 1, 64, 128, [n, keep + 1, 5], keep, min(50, keep), RANDOM, seed=n)


def test_evict_max_len_and_nothing_to_do(vq):
    evict(vq, 2, 64, 32, [300, 100], 50, 10, RANDOM, seed=4, max_len=200)
    evict(vq, 2, 64, 32, [300, 100], 300, 10, RANDOM, seed=5)
    evict(vq, 2, 64, 32, [300, 100], 50, 10, RANDOM, seed=6, max_len=50)


def test_evict_then_attend(vq):
    """Attention over what stays equals attention over those tokens alone."""
    rng = np.random.default_rng(15)
    lens, keep, recent = [200, 90], 40, 8
    cache, table, t = filled(vq, rng, lens, 2, 64, 32)
    q, q64 = heads(rng, 2, 4, 64, "bf16")
    pool = host_pool(cache)
    vq.kv4_evict(cache, t, ints(lens), ints(lens), keep=keep, recent=recent)
    pool.evict(table, lens, lens, keep, recent)
    ref, _, _, mag, vsum, smag = oa.attend_ref(q64, pool, table, [keep, keep], 0.125)
    out = vq.kv4_attend(q, cache, t, ints([keep, keep]))
    check(out, ref, oa.prompt_bound(ref, mag, vsum, smag.T, 64, keep, "bf16", "fp16", 2.0 ** -11), "after eviction")
