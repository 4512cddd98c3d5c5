"""Attention at the ends of its range: scores far beyond what a 24-bit product
resolves, and weight spread thinly over very many tokens."""
import numpy as np
import pytest

import oracle.attention as oa
from attntest import block_table, check, ints, new_cache, offsets, torch_type
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


def stored(vq, k, v, lens, page, seed):
    """A cache of the packed rows; its block table on the host and the GPU, and
    the keys and values that it stands for, float64."""
    import torch
    per = max(1, -(-max(lens) // page))
    table = block_table(np.random.default_rng(seed), len(lens), per, len(lens) * per)
    cache = new_cache(vq, table.size, page, k.shape[1], k.shape[2])
    _, cu = offsets(lens)
    t = torch.from_numpy(table).cuda()
    vq.kv4_append(cache, k, v, cu, t)
    k, v = vq.kv4_read(cache, cu, t, sum(lens), dtype=torch.float32)
    return cache, table, t, k.double().cpu().numpy(), v.double().cpu().numpy()


def one_query(q, k, v, lens, scale):
    """out and lse [B, Hq], the weights [Hq, T], sum_j p_j |v_j| and sum_j |v_j|
    of one query a sequence over packed keys and values, float64."""
    hq, g = q.shape[1], q.shape[1] // k.shape[1]
    out, mag, vsum = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, p, at = np.zeros(q.shape[:2]), np.zeros((hq, k.shape[0])), 0
    for b, n in enumerate(lens):
        for h in range(hq):
            kk, vv = k[at:at + n, h // g], v[at:at + n, h // g]
            p[h, at:at + n], lse[b, h] = oa.softmax_rows(kk @ q[b, h] * scale)
            out[b, h], mag[b, h], vsum[b, h] = p[h, at:at + n] @ vv, p[h, at:at + n] @ np.abs(vv), np.abs(vv).sum(0)
        at += n
    return out, lse, p, mag, vsum


def signs(rng, n, h, d, kind, size):
    """+-size, [n, h, d]: products of powers of two, so scores are exact in fp32."""
    import torch
    x = torch.from_numpy((rng.integers(0, 2, (n, h, d)) * 2.0 - 1.0) * size).to(torch_type(kind))
    return x.cuda(), x.double().numpy()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[200, 33], [1500, 70]])
def test_attend_scores_beyond_products(vq, lens, d, kind):
    """Scores of 2^33 and more: the keys are a step times a code plus a minimum,
    all with few bits, so that scores are exact in fp32 and equal ones tie; the
    result is the mean over the largest."""
    import torch
    rng = np.random.default_rng(d)
    k, _ = signs(rng, sum(lens), 2, d, "fp32", 16384.0)
    v = torch.from_numpy(rng.standard_normal((sum(lens), 2, d)).astype(np.float32)).cuda()
    cache, table, t, k64, v64 = stored(vq, k, v, lens, 64, d)
    q, q64 = signs(rng, len(lens), 6, d, kind, 16384.0)
    ref, lref, p, mag, vsum = one_query(q64, k64, v64, lens, 1.0)
    bound = oa.prompt_bound(ref, mag, vsum, np.zeros((6, len(lens))), d, max(lens), kind, "fp16", 2.0 ** -11)
    cache.weights.zero_()
    for weigh in (False, True):
        out, lse = vq.kv4_attend(q, cache, t, ints(lens), scale=1.0, add_weights=weigh, return_lse=True)
        check(out, ref, bound, "out")
        check(lse, lref, oa.lse_bound(lref, np.zeros_like(lref), d, max(lens)), "lse")
    got, at = cache.weights.cpu().numpy(), 0
    for b, n in enumerate(lens):
        slots = np.arange(n)
        w = got[table[b, slots // 64], :, slots % 64]
        want = p[:, at:at + n].reshape(2, 3, n).sum(1).T
        np.testing.assert_allclose(w, want, rtol=2.0 ** -19, atol=0)
        at += n


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,klens", [([150, 33], [150, 33]), ([60], [2100])])
def test_prompt_scores_beyond_products(vq, lens, klens, d, kind):
    """The same for prompts, with their keys in one piece and in several:
    scores are multiples of 2^30 up to 2^38."""
    import torch
    rng = np.random.default_rng(d)
    (cu, cu_d), (ck, ck_d) = offsets(lens), offsets(klens)
    q, q64 = signs(rng, sum(lens), 4, d, kind, 32768.0)
    k, k64 = signs(rng, sum(klens), 2, d, kind, 32768.0)
    v = torch.from_numpy(rng.standard_normal((sum(klens), 2, d)).astype(np.float32)).to(torch_type(kind))
    ref, lref, mag, vsum, _ = oa.prompt_ref(q64, k64, v.double().numpy(), cu, ck, 1.0, True)
    zero = np.zeros_like(lref)
    out, lse = vq.attn_prompt(q, k, v.cuda(), cu_d, ck_d, scale=1.0, return_lse=True)
    check(lse, lref, oa.lse_bound(lref, zero, d, max(klens)), "lse")
    check(out, ref, oa.prompt_bound(ref, mag, vsum, zero, d, max(klens), kind), "out")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,klens", [([150, 33], [150, 33]), ([900], [40])])
def test_gathered_weights_of_scores_beyond_products(vq, lens, klens, d, kind):
    """And for the weights their keys gather: exp(s - lse) of a score and an
    lse that are both multiples of large powers of two."""
    rng = np.random.default_rng(d)
    (cu, cu_d), (ck, ck_d) = offsets(lens), offsets(klens)
    q, q64 = signs(rng, sum(lens), 4, d, kind, 32768.0)
    k, k64 = signs(rng, sum(klens), 2, d, kind, 32768.0)
    _, lse = vq.attn_prompt(q, k, k, cu_d, ck_d, scale=1.0, return_lse=True)
    w = vq.attn_prompt_weights(q, k, lse, cu_d, ck_d, scale=1.0)
    want, _ = oa.prompt_weights_ref(q64, k64, lse.double().cpu().numpy(), cu, ck, 1.0, True, 0)
    assert want.max() >= 1.0
    check(w, want, want * ((2 * max(lens) + 8) * 2.0 ** -24 + 2.0 ** -20), "weights")


def sinks(rng, n, d, at, below, kind):
    """Keys and values of n tokens for a query of ones with scale 1 / d: every
    32nd token from `at` on has score 0 and value 0, the others' scores lie
    `below` under that (spread 0.5) and their values about 1000."""
    import torch
    k = torch.from_numpy((rng.standard_normal((n, 1, d)) * (0.5 * d ** 0.5) - below).astype(np.float32))
    v = torch.from_numpy((1000.0 + 100.0 * rng.standard_normal((n, 1, d))).astype(np.float32))
    k[at::32] = 0.0
    v[at::32] = 0.0
    return k.to(torch_type(kind)).cuda(), v.to(torch_type(kind)).cuda()


def thin(ref, mag, vsum, smag, largest, d, n, kind, **kw):
    """prompt_bound where the largest probability of the row is known: what is
    below fp16's normal range is off by 2^-32 of it."""
    return oa.prompt_bound(ref, mag, vsum * largest, smag, d, n, kind, **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d,n", [(64, 20000), (128, 10003), (256, 9001), (64, 1000), (256, 777)])
@pytest.mark.parametrize("below", [17.0, 18.5])
def test_attend_thin_weights(vq, d, n, kind, below):
    """Some slots take nearly all the weight and give nothing; the result is
    what the others, each of 2^-24 of the largest or less, add up to."""
    import torch
    rng = np.random.default_rng(d)
    for at in (0, 31):
        k, v = sinks(rng, n, d, at, below, "fp32")
        cache, table, t, k64, v64 = stored(vq, k, v, [n], 256, d)
        q = torch.ones((1, 3, d), dtype=torch_type(kind), device="cuda")
        ref, lref, p, mag, vsum = one_query(np.ones((1, 3, d)), k64, v64, [n], 1.0 / d)
        smag = np.full((1, 3), np.abs(k64).sum(2).max() / d)
        bound = thin(ref, mag, vsum, smag.T, p.max(), d, n, kind, p_kind="fp16", v_round=2.0 ** -11)
        for weigh in (False, True):
            cache.weights.zero_()
            out, lse = vq.kv4_attend(q, cache, t, ints([n]), scale=1.0 / d, add_weights=weigh, return_lse=True)
            check(out, ref, bound, f"out, weigh {weigh}, at {at}")
            check(lse, lref, oa.lse_bound(lref, smag, d, n), "lse")
        slots = np.arange(n)
        w = cache.weights.double().cpu().numpy()[table[0, slots // 256], 0, slots % 256]
        want = p.sum(0)
        rel = 2.0 * (smag[0, 0] * ((d + 8) * 2.0 ** -24 + 2.0 ** -22) + (n + 8) * 2.0 ** -24) + 2.0 ** -20
        assert (np.abs(w - want) <= rel * want).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d,n", [(64, 20000), (128, 10003), (256, 9001), (64, 1000), (256, 777)])
@pytest.mark.parametrize("below", [17.0, 18.5])
def test_prompt_thin_weights(vq, d, n, kind, below):
    """The same for prompts: a few rows against keys in pieces, and rows whose
    keys are taken in one."""
    import torch
    rng = np.random.default_rng(d)
    for at, nq in ((0, 3), (31, 700)):
        k, v = sinks(rng, n, d, at, below, kind)
        cu, cu_d = offsets([nq])
        ck, ck_d = offsets([n])
        q = torch.ones((nq, 2, d), dtype=torch_type(kind), device="cuda")
        out, lse = vq.attn_prompt(q, k, v, cu_d, ck_d, scale=1.0 / d, causal=False, return_lse=True)
        assert torch.equal(out[1:], out[:1].expand(nq - 1, -1, -1)) and torch.equal(lse[:, 1:], lse[:, :1].expand(-1, nq - 1))
        k64, v64 = k.double().cpu().numpy(), v.double().cpu().numpy()
        ref, lref, p, mag, vsum = one_query(np.ones((1, 2, d)), k64, v64, [n], 1.0 / d)
        smag = np.full((2, 1), np.abs(k64).sum(2).max() / d)
        if kind == "fp16":
            bound = thin(ref, mag, vsum, smag, p.max(), d, n, kind)
        else:
            bound = oa.prompt_bound(ref, mag, vsum * 0.0, smag, d, n, kind)  # bf16 rounds relatively all the way down
        check(out[:1], ref, bound, "out")
        check(lse[:, :1], lref.T, oa.lse_bound(lref.T, smag, d, n), "lse")
