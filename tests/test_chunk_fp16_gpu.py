"""kv4_attend_chunk's fp16 results are as near as their own rounding and that of
the values leave them: keys and probabilities rounded to fp16 would show."""
import numpy as np
import pytest

import oracle.attention as oa
from attntest import check, heads, ints, offsets
from test_chunk_gpu import ROUND, filled, vq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(None, 0), (700, 20)])
@pytest.mark.parametrize("lq,lens", [([4, 2], [5000, 1300]), ([4, 4], [400, 90]), ([300, 70], [2500, 300]),
                                     ([300, 1, 3], [4000, 1500, 37])])
@pytest.mark.parametrize("d,hq,hkv", [(64, 6, 2), (128, 8, 2), (256, 4, 1)])
def test_fp16_errors(vq, d, hq, hkv, lq, lens, window, sinks):  # noqa: F811
    rng = np.random.default_rng(d + sum(lq))
    cache, table, k64, v64 = filled(vq, rng, lens, 64, hkv, d)
    q, q64 = heads(rng, sum(lq), hq, d, "fp16")
    c, cu = offsets(lq)
    out, lse = vq.kv4_attend_chunk(q, cache, table, ints(lens), cu, window=window, sinks=sinks, max_q=max(lq), return_lse=True)
    ref, lref, mag, vsum, _ = oa.chunk_ref(q64, k64, v64, c, lens, d ** -0.5, window or 0, sinks)
    # Minimum, steps and centred codes are summed apart: with the group's largest |k| they are below 3.3 times it (the
    # minimum once, 8 and up to 8 steps of two fifteenths).  The sums of queries are held to 2^-22, and so are
    # probabilities, in two parts.
    n, kept = max(lens), 2.0 ** -22
    top = np.abs(k64).reshape(len(k64), hkv, -1, 32).max((0, 1, 3))
    smag = (3.3 * d ** -0.5 * np.abs(q64).reshape(*q64.shape[:2], -1, 32).sum(-1) @ top).T
    check(lse, lref, oa.lse_bound(lref, smag, d, n, kept), "lse")
    check(out, ref, oa.prompt_bound(ref, mag, vsum, smag, d, n, "fp16", "fp32", ROUND + kept, kept), "out")
    # As a whole: a rounding to fp16 is uniform within half a step, so at most 2^-11 / sqrt(3) of a value as a root mean
    # square.  Two of them, independent: the result's, and the values', which the probabilities weight as they do the
    # values of mean zero themselves, so it is the same part of the result.  (Rounded keys and probabilities: 4.9e-4.)
    err = out.double().cpu().numpy() - ref
    assert np.sqrt((err ** 2).mean()) <= np.sqrt((ref ** 2).mean()) * 2.0 ** -11 * (2.0 / 3.0) ** 0.5
