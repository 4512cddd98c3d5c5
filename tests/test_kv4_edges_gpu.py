"""The 4-bit cache where its format ends: groups at the saturation limits, and
what stands in them read by the decode kernel."""
import numpy as np
import pytest

import oracle.attention as oa
from attntest import check, heads, host_pool, ints, new_cache, offsets, torch_type
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_append_beside_saturation(vq, kind):
    """Groups whose smallest value rounds up to the limit, or nearly, with
    values beyond it: the codes are those of the saturated values."""
    import torch
    rng = np.random.default_rng(1)
    rows = []
    for low in (32767.5, 32764.0, 32760.0, 32753.0, 32752.0, 32750.0, 32700.0, 32640.0, 32000.0):
        for big in (np.inf, 65000.0, 40000.0, 32769.0, 32768.0):
            for end in (1.0, -1.0):
                x = np.full(64, low) + rng.random(64) * (32768.0 - low)
                x[rng.integers(0, 64, 20)] = big
                x[::9] = low
                rows.append(end * x)
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(torch_type(kind)).view(len(rows), 1, 64)
    cache = new_cache(vq, 3, 32, 1, 64)
    pool = host_pool(cache)
    cu, cu_d = offsets([len(rows)])
    vq.kv4_append(cache, x.cuda(), x.cuda(), cu_d, ints([[0, 2, 1]]))
    f = x.float().numpy()
    pool.append(f, f, cu, np.array([[0, 2, 1]], np.int32), [0])
    np.testing.assert_array_equal(cache.codes.cpu().numpy(), pool.codes)
    np.testing.assert_array_equal(cache.scales.cpu().numpy().view(np.uint16), pool.scales.view(np.uint16))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_over_saturated_values(vq, d, kind):
    """Groups over the whole range have the step 4368, and 15 * 4368 is beyond
    fp16: a value is finite because the minimum is added before it is rounded."""
    import torch
    rng = np.random.default_rng(d)
    n, page = 90, 32
    k, _ = heads(rng, n, 2, d, "fp32")
    v = torch.from_numpy((rng.choice([-1.0, 1.0], (n, 2, d)) * rng.choice([3.0, 3e4, 7e4], (n, 2, d))).astype(np.float32))
    v[:, :, ::32], v[:, :, 1::32] = 1e5, -1e5
    cache = new_cache(vq, 3, page, 2, d)
    _, cu_d = offsets([n])
    table = np.array([[1, 0, 2]], np.int32)
    t = torch.from_numpy(table).cuda()
    vq.kv4_append(cache, k, v.cuda(), cu_d, t)
    pool = host_pool(cache)
    assert np.nanmax(pool.scales[:, 1, ..., :4].astype(np.float64)) == 4368.0
    q, q64 = heads(rng, 1, 6, d, kind)
    ref, lref, _, mag, vsum, smag = oa.attend_ref(q64, pool, table, [n], d ** -0.5)
    bound = oa.prompt_bound(ref, mag, vsum, smag.T, d, n, kind, "fp16", 2.0 ** -11)
    for weigh in (False, True):
        out = vq.kv4_attend(q, cache, t, ints([n]), add_weights=weigh)
        check(out, ref, bound, "out")


def test_evict_moves_in_rounds(vq):
    """More rows and moves than one launch has workgroups for: each takes its
    moves in rounds.  One sequence is cut, among hundreds of empty ones; the
    pool equals that of the sequence cut alone."""
    import torch
    hkv, page, keep, n, others = 32, 1024, 16400, 32700, 544
    gen = torch.Generator(device="cuda").manual_seed(3)
    pages = 32
    codes = torch.randint(0, 256, (pages, 2, hkv, page * 32), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.rand((pages, 2, hkv, page // 4, 2, 8), device="cuda", generator=gen).half()
    weights = torch.rand((pages, hkv, page), device="cuda", generator=gen)
    weights[16:] += 1.0  # nearly all that stay lie above keep
    pos = torch.randint(0, 1000, (pages, hkv, page), dtype=torch.int32, device="cuda", generator=gen)
    both = []
    for seqs in (1, others):
        cache = vq.KV4Cache.from_buffers(codes.clone(), scales.clone(), weights.clone(), pos.clone())
        table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(seqs, 1)
        lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        lens[-1] = n
        vq.kv4_evict(cache, table, lens, torch.full_like(lens, 5000), keep=keep, recent=0, max_len=32768)
        both.append(cache)
    one, many = both
    assert not torch.equal(one.pos, pos)
    assert torch.equal(one.codes, many.codes) and torch.equal(one.scales, many.scales)
    assert torch.equal(one.weights, many.weights) and torch.equal(one.pos, many.pos)


@pytest.mark.parametrize("d,hq,hkv", [(64, 3, 1), (128, 40, 2), (256, 4, 2)])
def test_weights_with_a_wide_table(vq, d, hq, hkv):
    """Weights added over a table far wider than the pool: the workspace is the
    pool's, results and weights are those of a table that just fits; more than
    64 sequences, empty ones among them."""
    import torch
    rng = np.random.default_rng(d)
    page = 32
    lens = [int(n) for n in rng.integers(0, 70, 90)]
    lens[3], lens[60], lens[70], lens[89] = 0, 1200, 0, 333
    used = [-(-n // page) for n in lens]
    order = rng.permutation(sum(used))
    table = np.zeros((90, 4000), np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    _, cu_d = offsets(lens)
    k, _ = heads(rng, sum(lens), hkv, d, "bf16")
    v, _ = heads(rng, sum(lens), hkv, d, "bf16")
    q, _ = heads(rng, 90, hq, d, "bf16")
    cache = new_cache(vq, sum(used), page, hkv, d)
    wide = torch.from_numpy(table).cuda()
    narrow = wide[:, :max(used)].contiguous()
    vq.kv4_append(cache, k, v, cu_d, narrow)
    results = []
    for t in (narrow, wide):
        cache.weights.zero_()
        need = vq.kv4_attend_workspace_size(cache, 90, hq, t.shape[1] * page, True)
        assert need < vq.kv4_attend_workspace_size(cache, 90, hq, 2000, False) + sum(used) * page * hq * 4 + 90 * hq * 8 + 1024
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse = vq.kv4_attend(q, cache, t, ints(lens), add_weights=True, return_lse=True, workspace=ws)
        results.append((out, lse, cache.weights.clone()))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    # every head of a sequence that is not empty hands out a weight of one
    total = results[0][2].double().sum().item()
    np.testing.assert_allclose(total, hq * sum(n > 0 for n in lens), rtol=1e-5)


def attend_case(vq, kind, hq, hkv, d, page, lens, seed):
    """Results against the oracle, with and without weights."""
    import torch
    rng = np.random.default_rng(seed)
    per = -(-max(lens) // page)
    table = rng.permutation(len(lens) * per).reshape(len(lens), per).astype(np.int32)
    cache = new_cache(vq, table.size, page, hkv, d)
    _, cu_d = offsets(lens)
    k, _ = heads(rng, sum(lens), hkv, d, "fp32", 1.0, 1.5)
    v, _ = heads(rng, sum(lens), hkv, d, "fp32")
    t = torch.from_numpy(table).cuda()
    vq.kv4_append(cache, k, v, cu_d, t)
    q, q64 = heads(rng, len(lens), hq, d, kind)
    ref, lref, _, mag, vsum, smag = oa.attend_ref(q64, host_pool(cache), table, lens, d ** -0.5)
    bound = oa.prompt_bound(ref, mag, vsum, smag.T, d, max(lens), kind, "fp16", 2.0 ** -11)
    for weigh in (False, True):
        out, lse = vq.kv4_attend(q, cache, t, ints(lens), add_weights=weigh, return_lse=True)
        check(out, ref, bound, f"out, weigh {weigh}")
        check(lse, lref, oa.lse_bound(lref, smag, d, max(lens)), "lse")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (20, 1)])
def test_attend_wide_heads_in_shares(vq, hq, hkv, kind):
    """Heads of 256 beyond what one workgroup takes whole: rows cut over
    several shares, short and empty ones beside them, a group of more than 16."""
    attend_case(vq, kind, hq, hkv, 256, 96, [2500, 3, 0, 129, 1100], seed=hq)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("n,hkv,d", [(1024, 1, 64), (1025, 1, 64), (1024, 129, 64), (40, 129, 64), (1024, 2, 128),
                                     (1025, 2, 128), (768, 1, 256), (769, 1, 256)])
def test_attend_where_its_form_changes(vq, n, hkv, d, kind):
    """Both sides of the length up to which a workgroup takes a row whole, and
    more rows than CUs."""
    need = vq.kv4_attend_workspace_size(vq.KV4Cache(1, 32, hkv, d), 2, hkv, n)
    assert (need == 0) == (n in (40, 768, 1024))
    attend_case(vq, kind, hkv, hkv, d, 32, [n, 7], seed=n + hkv)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[60, 60], [1500, 60]])
def test_attend_query_that_is_not_finite(vq, lens, d, bad):
    """It reaches its own head and no other: sequences and key/value heads
    beside it keep their bits, query heads of its group their results within
    the bound (they share its reference maximum's updates)."""
    import torch
    rng = np.random.default_rng(d)
    page, per = 64, -(-max(lens) // 64)
    table = rng.permutation(2 * per).reshape(2, per).astype(np.int32)
    cache = new_cache(vq, table.size, page, 2, d)
    _, cu_d = offsets(lens)
    k, _ = heads(rng, sum(lens), 2, d, "bf16")
    v, _ = heads(rng, sum(lens), 2, d, "bf16")
    t = torch.from_numpy(table).cuda()
    vq.kv4_append(cache, k, v, cu_d, t)
    q, _ = heads(rng, 2, 4, d, "bf16")
    want, lse = vq.kv4_attend(q, cache, t, ints(lens), return_lse=True)
    ref, _, _, mag, vsum, smag = oa.attend_ref(q.double().cpu().numpy(), host_pool(cache), table, lens, d ** -0.5)
    bound = oa.prompt_bound(ref, mag, vsum, smag.T, d, max(lens), "bf16", "fp16", 2.0 ** -11)
    q[0, 1, 5] = bad
    for weigh in (False, True):
        got, l2 = vq.kv4_attend(q, cache, t, ints(lens), add_weights=weigh, return_lse=True)
        assert not bool(torch.isfinite(got[0, 1]).any()) and not bool(torch.isfinite(l2[0, 1]))
        check(got[0, :1], ref[0, :1], bound[0, :1], "the head beside it")
        check(got[0, 2:], ref[0, 2:], bound[0, 2:], "the other key/value head")
        check(got[1], ref[1], bound[1], "the other sequence")
        if not weigh:
            assert torch.equal(got[0, 2:], want[0, 2:]) and torch.equal(got[1], want[1])
            assert torch.equal(l2[0, 2:], lse[0, 2:]) and torch.equal(l2[1], lse[1])
