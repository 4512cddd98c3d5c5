"""One workspace, sized for the largest call, through calls of every form."""
import numpy as np
import pytest

from attntest import heads, ints, offsets
from test_chunk_gpu import filled, vq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hkv", [(64, 6, 2), (128, 32, 8), (256, 4, 2)])
def test_calls_share_a_workspace(vq, d, hq, hkv):  # noqa: F811
    import torch
    rng = np.random.default_rng(d)
    capacity, largest = 3520, 2100
    cache, table, _, _ = filled(vq, rng, [capacity], 32, hkv, d)
    q, _ = heads(rng, largest, hq, d, "bf16")
    size = vq.kv4_attend_chunk_workspace_size(cache, 1, hq, largest, capacity)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    for tq, n in ((largest, capacity), (700, 3300), (300, 900), (64, 3100), (5, 3500), (1, 40), (2000, 2000)):
        cu = offsets([tq])[1]
        for max_len in (None, n):
            want = vq.kv4_attend_chunk(q[:tq], cache, table, ints([n]), cu, max_len=max_len, return_lse=True)
            got = vq.kv4_attend_chunk(q[:tq], cache, table, ints([n]), cu, max_len=max_len, return_lse=True, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (tq, n, max_len)
