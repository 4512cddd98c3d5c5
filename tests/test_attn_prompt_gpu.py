"""attn_prompt and attn_prompt_weights against the float64 oracle, within the
bounds that the oracle derives from their roundings."""
import numpy as np
import pytest

import oracle.attention as oa
from attntest import check, heads, ints, offsets
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


def one(vq, kind, hq, hkv, d, lens, klens=None, causal=True, scale=None, spread=1.0, seed=0, fused=False, last=(0, 1, 50)):
    import torch
    rng = np.random.default_rng(seed)
    scale = d ** -0.5 if scale is None else scale
    cu, cu_d = offsets(lens)
    ck, ck_d = offsets(lens if klens is None else klens)
    q, q64 = heads(rng, cu[-1], hq, d, kind, spread)
    k, k64 = heads(rng, ck[-1], hkv, d, kind, spread, 1.0)
    v, v64 = heads(rng, ck[-1], hkv, d, kind)
    if fused:
        q, k, v = torch.cat([q, k, v], 1).split([hq, hkv, hkv], 1)
    out, lse = vq.attn_prompt(q, k, v, cu_d, None if klens is None else ck_d, scale=scale, causal=causal, return_lse=True)
    ref, lref, mag, vsum, smag = oa.prompt_ref(q64, k64, v64, cu, ck, scale, causal)
    n = max([0, *np.diff(ck)])
    check(lse, lref, oa.lse_bound(lref, smag, d, n), "lse")
    check(out, ref, oa.prompt_bound(ref, mag, vsum, smag, d, n, kind), "out")
    lse64 = lse.double().cpu().numpy()
    for few in last:
        w = vq.attn_prompt_weights(q, k, lse, cu_d, None if klens is None else ck_d, scale=scale, causal=causal, last=few)
        wref, wmag = oa.prompt_weights_ref(q64, k64, lse64, cu, ck, scale, causal, few)
        nq = max([0, *np.diff(cu)]) * (hq // hkv)
        top = np.abs(lse64[np.isfinite(lse64)]).max(initial=0.0)
        rel = wmag * ((d + 8) * 2.0 ** -24 + 2.0 ** -22) + (top + 1) * 2.0 ** -21 + (nq + 8) * 2.0 ** -24
        check(w, wref, wref * rel * 1.1 + 2.0 ** -100, f"weights of the last {few}")
    return out, lse


EDGES = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d", [(3, 1, 64), (4, 2, 128), (2, 1, 256)])
def test_lengths_around_tiles(vq, hq, hkv, d, causal, kind):
    one(vq, kind, hq, hkv, d, EDGES, causal=causal, seed=d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (9, 3), (16, 2), (17, 1), (20, 4)])
def test_head_groups(vq, hq, hkv):
    one(vq, "bf16", hq, hkv, 64, [70, 1, 150], seed=hq, fused=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_and_rows_without_keys(vq, d, causal):
    """Keys longer and shorter than the queries, none at all, no queries."""
    one(vq, "fp16", 4, 2, d, [40, 100, 33, 7, 0, 130], [300, 60, 0, 8, 50, 129], causal=causal, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d", [(3, 1, 64), (4, 2, 128), (2, 1, 256)])
def test_few_rows_against_many_keys(vq, hq, hkv, d, kind):
    """Keys in pieces: the call asks for a workspace; rows of long, short and
    no keys side by side; the workspace may hold anything."""
    import torch
    from compressed_index_matmul_amd.attention import AttnBatch
    b = AttnBatch(1, hq, hkv, d, 4, 218, 3030, 1, 0.1, 0, None, None)
    need = vq.lib().attn_prompt_workspace_size(b)
    assert need > 0
    lens, klens = [130, 1, 80, 7], [2500, 300, 230, 0]
    for causal in (True, False):
        out, lse = one(vq, kind, hq, hkv, d, lens, klens, causal=causal, seed=d, last=(0, 20))
    rng = np.random.default_rng(d)
    cu, cu_d = offsets(lens)
    ck, ck_d = offsets(klens)
    q, _ = heads(rng, cu[-1], hq, d, kind)
    k, _ = heads(rng, ck[-1], hkv, d, kind)
    want, l1 = vq.attn_prompt(q, k, k, cu_d, ck_d, return_lse=True)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got, l2 = vq.attn_prompt(q, k, k, cu_d, ck_d, return_lse=True, workspace=ws)
    assert torch.equal(got, want) and torch.equal(l1, l2)
    with pytest.raises(vq.VQError) as e:
        vq.attn_prompt(q, k, k, cu_d, ck_d, workspace=ws[:need - 16])
    assert e.value.status == -8
    # a value that is not finite, in the last piece, reaches the queries that see it and no other
    v = k.clone()
    v[2500 - 100, 0, 7] = float("inf")
    got = vq.attn_prompt(q, k, v, cu_d, ck_d)
    sees = 130 - 100  # the first query of the first sequence that sees that key
    group = hq // hkv
    assert torch.equal(got[:sees], vq.attn_prompt(q, k, k, cu_d, ck_d)[:sees])
    assert bool((got[sees:130, :group, 7] == float("inf")).all()) and bool(torch.isfinite(got[sees:130, :, 8:]).all())


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (2, 2, 128), (1, 1, 256)])
def test_many_tiles(vq, hq, hkv, d):
    """Long enough for dozens of tiles, with keys whose scores grow along the
    sequence, so that the running maximum moves all the time."""
    import torch
    rng = np.random.default_rng(d)
    n = 1500
    cu, cu_d = offsets([n])
    ramp = torch.linspace(0.1, 6.0, n)[:, None, None]
    q, q64 = heads(rng, n, hq, d, "bf16")
    k = (torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32)) * ramp).bfloat16()
    v, v64 = heads(rng, n, hkv, d, "bf16")
    k64, k = k.double().numpy(), k.cuda()
    out, lse = vq.attn_prompt(q, k, v, cu_d, return_lse=True)
    ref, lref, mag, vsum, smag = oa.prompt_ref(q64, k64, v64, cu, cu, d ** -0.5, True)
    check(lse, lref, oa.lse_bound(lref, smag, d, n), "lse")
    check(out, ref, oa.prompt_bound(ref, mag, vsum, smag, d, n, "bf16"), "out")


def test_empty_batches(vq):
    import torch
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    for cu in ([0], [0, 0, 0]):
        out, lse = vq.attn_prompt(q, k, k, ints(cu), return_lse=True)
        assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
        assert vq.attn_prompt_weights(q, k, lse, ints(cu)).shape == (2, 0)
    # queries without any key
    q = torch.ones((5, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = vq.attn_prompt(q, k, k, ints([0, 5]), ints([0, 0]), return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_large_scores(vq):
    """Scores in the thousands: one key takes almost all, nothing overflows."""
    one(vq, "bf16", 2, 2, 128, [150, 64], spread=12.0, scale=1.0, seed=5)
    one(vq, "fp16", 2, 1, 64, [99], spread=30.0, scale=2.0, seed=6)


def test_small_scale(vq):
    one(vq, "bf16", 2, 1, 64, [150], scale=1e-6, seed=7)


def test_strides(vq):
    """Head-major storage, odd row strides, a slice of a fused row: the results
    of contiguous inputs, bit for bit."""
    import torch
    rng = np.random.default_rng(3)
    cu, cu_d = offsets([70, 33])
    q, _ = heads(rng, 103, 6, 128, "bf16")
    k, _ = heads(rng, 103, 2, 128, "bf16")
    v, _ = heads(rng, 103, 2, 128, "bf16")
    want, lse = vq.attn_prompt(q, k, v, cu_d, return_lse=True)
    wref = vq.attn_prompt_weights(q, k, lse, cu_d)

    def head_major(x):
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    def odd_rows(x):
        wide = torch.full((x.shape[0], x.shape[1] + 3, x.shape[2] + 8), float("nan"), dtype=x.dtype, device="cuda")
        part = wide[:, 1:1 + x.shape[1], 8:]
        part.copy_(x)
        return part

    for form in (head_major, odd_rows):
        got, l2 = vq.attn_prompt(form(q), form(k), form(v), cu_d, return_lse=True)
        assert torch.equal(got, want) and torch.equal(l2, lse)
        assert torch.equal(vq.attn_prompt_weights(form(q), form(k), lse, cu_d), wref)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_other_rows_do_not_reach_a_sequence(vq, d, bad):
    """Sequences next to rows of NaN or infinities in the pack."""
    import torch
    rng = np.random.default_rng(4)
    lens = [37, 50, 90, 3]
    cu, cu_d = offsets(lens)
    q, _ = heads(rng, cu[-1], 4, d, "bf16")
    k, _ = heads(rng, cu[-1], 2, d, "bf16")
    v, _ = heads(rng, cu[-1], 2, d, "bf16")
    want, lse = vq.attn_prompt(q, k, v, cu_d, return_lse=True)
    wref = vq.attn_prompt_weights(q, k, lse, cu_d)
    for b in (0, 2):
        for x in (q, k, v):
            x[cu[b]:cu[b + 1]] = bad
    got, l2 = vq.attn_prompt(q, k, v, cu_d, return_lse=True)
    w = vq.attn_prompt_weights(q, k, lse, cu_d)
    for b in (1, 3):
        rows = slice(cu[b], cu[b + 1])
        assert torch.equal(got[rows], want[rows]) and torch.equal(l2[:, rows], lse[:, rows])
        assert torch.equal(w[:, rows], wref[:, rows])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_masked_places_hold_anything(vq, d, kind, bad):
    """A non-finite value or key reaches the queries that see it and no other,
    within the same tile too; the channels beside it stay as they were."""
    import torch
    rng = np.random.default_rng(d)
    n, keys = 150, (149, 77, 64, 40, 5)
    cu, cu_d = offsets([n])
    q, _ = heads(rng, n, 2, d, kind)
    k, _ = heads(rng, n, 1, d, kind)
    v, _ = heads(rng, n, 1, d, kind)
    want, lse = vq.attn_prompt(q, k, v, cu_d, return_lse=True)
    wref = vq.attn_prompt_weights(q, k, lse, cu_d)
    for j in keys:
        v2 = v.clone()
        v2[j, 0, 3] = v2[j, 0, d - 1] = bad
        got, l2 = vq.attn_prompt(q, k, v2, cu_d, return_lse=True)
        assert torch.equal(l2, lse)
        assert torch.equal(got[:j], want[:j]), j
        others = torch.ones(d, dtype=torch.bool, device="cuda")
        others[3] = others[d - 1] = False
        assert torch.equal(got[j:, :, others], want[j:, :, others]), j
        hit = got[j:, :, ~others].float()
        assert bool((torch.isnan(hit) if bad != bad else hit == bad).all()), j
        k2 = k.clone()
        k2[j] = bad
        got, l2 = vq.attn_prompt(q, k2, v, cu_d, return_lse=True)
        assert torch.equal(got[:j], want[:j]) and torch.equal(l2[:, :j], lse[:, :j]), j
        if j == n - 1:  # the weights of the keys before it, over the queries before it
            w = vq.attn_prompt_weights(q[:j], k2[:j], lse[:, :j].contiguous(), ints([0, j]))
            assert bool(torch.isfinite(w).all())


def test_weights_accumulate_and_sum(vq):
    import torch
    rng = np.random.default_rng(8)
    cu, cu_d = offsets([130, 17])
    q, _ = heads(rng, 147, 6, 64, "bf16")
    k, _ = heads(rng, 147, 3, 64, "bf16")
    _, lse = vq.attn_prompt(q, k, k, cu_d, return_lse=True)
    w = vq.attn_prompt_weights(q, k, lse, cu_d)
    # every query gives each head a total of one
    np.testing.assert_allclose(w[:, :130].sum(1).cpu().numpy(), 2 * 130, rtol=1e-5)
    twice = w.clone()
    out = vq.attn_prompt_weights(q, k, lse, cu_d, out=twice, accumulate=True)
    assert out.data_ptr() == twice.data_ptr() and torch.equal(twice, w + w)


def test_out_argument_and_other_stream(vq):
    import torch
    rng = np.random.default_rng(9)
    cu, cu_d = offsets([200, 60])
    q, _ = heads(rng, 260, 4, 128, "fp16")
    k, _ = heads(rng, 260, 4, 128, "fp16")
    want = vq.attn_prompt(q, k, k, cu_d)
    out = torch.full_like(want, 3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vq.attn_prompt(q, k, k, cu_d, out=out, stream=side)
    fresh = vq.attn_prompt(q, k, k, cu_d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want) and torch.equal(fresh, want)


def test_long_offsets(vq):
    """Rows far apart: element offsets beyond 2^31, byte offsets beyond 2^32."""
    import torch
    rng = np.random.default_rng(10)
    n, ts = 600, (1 << 22) - 8
    cu, cu_d = offsets([n - 40, 40])
    store = torch.empty(n * ts, dtype=torch.bfloat16, device="cuda")
    big = store.as_strided((n, 1, 64), (ts, 64, 1))
    small, _ = heads(rng, n, 1, 64, "bf16")
    big.copy_(small)
    want, lse = vq.attn_prompt(small, small, small, cu_d, return_lse=True)
    got, l2 = vq.attn_prompt(big, big, big, cu_d, return_lse=True)
    assert torch.equal(got, want) and torch.equal(l2, lse)
    assert torch.equal(vq.attn_prompt_weights(big, big, lse, cu_d), vq.attn_prompt_weights(small, small, lse, cu_d))


def test_inconsistent_offsets_stay_in_bounds(vq):
    """Offsets beyond the rows, negative or falling: clamped, no fault; a
    well-formed sequence among them keeps its result."""
    import torch
    rng = np.random.default_rng(11)
    q, _ = heads(rng, 100, 2, 64, "bf16")
    good = vq.attn_prompt(q[:50], q[:50], q[:50], ints([0, 50]))
    got = vq.attn_prompt(q, q, q, ints([0, 50, 4000]))
    assert torch.equal(got[:50], good)
    for cu in ([-5, 200], [0, 70, 30, 100], [100, 100, 0]):
        out, lse = vq.attn_prompt(q, q, q, ints(cu), return_lse=True)
        vq.attn_prompt_weights(q, q, lse, ints(cu))
    torch.cuda.synchronize()


def test_deterministic(vq):
    import torch
    rng = np.random.default_rng(12)
    cu, cu_d = offsets([513, 200])
    q, _ = heads(rng, 713, 8, 128, "bf16")
    k, _ = heads(rng, 713, 2, 128, "bf16")
    a, la = vq.attn_prompt(q, k, k, cu_d, return_lse=True)
    wa = vq.attn_prompt_weights(q, k, la, cu_d)
    for _ in range(3):
        b, lb = vq.attn_prompt(q, k, k, cu_d, return_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(wa, vq.attn_prompt_weights(q, k, la, cu_d))
