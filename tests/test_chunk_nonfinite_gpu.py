"""kv4_attend_chunk: rows of queries that are not finite are not finite, through
every kernel and join."""
import numpy as np
import pytest

import oracle.attention as oa
from attntest import check, heads, ints, offsets
from test_chunk_gpu import ROUND, filled, vq  # noqa: F401

pytestmark = pytest.mark.gpu

# (queries, slots, query heads of two key/value heads): whole row tiles of few rows and of many, few rows in shares joined
# a workgroup a row, the same beside a chunk in shares, and few rows in shares joined a row tile a workgroup
FORMS = [([7, 5], [200, 31], 4), ([150, 90], [200, 301], 4), ([7, 5], [5000, 3900], 4), ([150, 5], [5000, 2600], 4),
         ([5] * 28, [2500] + [90] * 27, 16)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("lq,lens,hq", FORMS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_are_not_finite_say_so(vq, d, lq, lens, hq, kind):  # noqa: F811
    """A NaN in a query makes its scores NaN.  An infinity of the sign that gives
    its first slot a score of plus infinity leaves inf - inf in the softmax."""
    rng = np.random.default_rng(d + len(lq))
    cache, table, k64, v64 = filled(vq, rng, lens, 32, 2, d)
    q, q64 = heads(rng, sum(lq), hq, d, kind)
    c, cu = offsets(lq)
    bad = np.zeros(q64.shape[:2], bool)
    first = np.concatenate([[0], np.cumsum(lens)])  # each sequence's first slot
    for i, (b, at) in enumerate([(0, 1), (0, 3), (1, 0), (1, 4), (0, lq[0] - 1), (1, lq[1] - 1)]):
        row, head, channel = c[b] + at, i % hq, 5 + i
        key = k64[first[b], head * 2 // hq, channel]
        assert key != 0.0
        q[row, head, channel] = float("nan") if i % 2 == 0 else float("inf") if key > 0 else float("-inf")
        bad[row, head] = True
    out, lse = vq.kv4_attend_chunk(q, cache, table, ints(lens), cu, max_len=max(lens), max_q=max(lq), return_lse=True)
    at = np.nonzero(bad)
    assert bool(out[at].isnan().all()), "results"
    assert bool(lse.T[at].isnan().all()), "lse"
    ref, lref, mag, vsum, smag = oa.chunk_ref(q64, k64, v64, c, lens, d ** -0.5)
    bound = oa.prompt_bound(ref, mag, vsum, smag, d, max(lens), kind, "fp16", ROUND, ROUND)
    rest = np.nonzero(~bad)
    check(out[rest], ref[rest], bound[rest], "finite queries")
    check(lse.T[rest], lref.T[rest], oa.lse_bound(lref, smag, d, max(lens), ROUND).T[rest], "their lse")
