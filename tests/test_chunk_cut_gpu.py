"""kv4_attend_chunk on very unequal lengths, row tiles whole and in shares, the
long sequence first and last."""
import numpy as np
import pytest

from test_chunk_gpu import run, vq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hkv,order", [(64, 64, 64, 1), (128, 32, 32, -1), (256, 32, 16, 1)])
@pytest.mark.parametrize("long", [1.0, 1.1])
def test_unequal_lengths(vq, d, hq, hkv, order, long):  # noqa: F811
    """384 row tiles and more.  They are whole as long as a tile meets at most
    5 own group hkv / 2^16 slots, own being the pairs of the chunks' own tokens."""
    kind = {64: "bf16", 128: "fp16", 256: "bf16"}[d]
    first = -(-384 * 256 // hq) // 2  # two chunks of these rows, and five tokens after many slots
    lq = [first + 200, 5, first]
    rest = (sum(lq) - lq[0]) / 2
    border = 5 * (lq[0] ** 2 + 2 * rest ** 2) / 2 * hq / 2 ** 16
    lens = [lq[0], int(border * long) // 2 * 2, lq[2]]
    run(vq, np.random.default_rng(d), lq[::order], lens[::order], hq, hkv, d, kind, page=64, max_len=max(lens), max_q=lq[0])
