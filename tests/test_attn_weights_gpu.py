"""attn_prompt_weights beside its numerics: what it leaves alone."""
import numpy as np
import pytest

from attntest import heads, offsets
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("lens,n,hq,pieces", [([600, 300], 1000, 4, True), ([3, 2], 20, 4, True), ([3, 2], 20, 2, False)])
def test_weights_of_uncovered_keys(vq, lens, n, hq, pieces, accumulate):
    """Keys past the last sequence keep what `out` holds, whether the queries
    are taken in pieces (a workspace) or not; the workspace may hold anything."""
    import torch
    from compressed_index_matmul_amd.attention import AttnBatch
    rng = np.random.default_rng(13)
    cu, cu_d = offsets(lens)
    q, _ = heads(rng, n, hq, 64, "bf16")
    k, _ = heads(rng, n, 2, 64, "bf16")
    _, lse = vq.attn_prompt(q[:cu[-1]], k[:cu[-1]], k[:cu[-1]], cu_d, return_lse=True)
    full = torch.zeros((hq, n), device="cuda")
    full[:, :cu[-1]] = lse
    want = vq.attn_prompt_weights(q[:cu[-1]], k[:cu[-1]], lse, cu_d)
    need = vq.lib().attn_prompt_weights_workspace_size(AttnBatch(1, hq, 2, 64, 2, n, n, 1, 0.125, 0, None, None), 0)
    assert (need > 0) == pieces
    out = torch.full((2, n), 5.0, device="cuda")
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    vq.attn_prompt_weights(q, k, full, cu_d, out=out, accumulate=accumulate, workspace=ws if need else None)
    assert bool((out[:, cu[-1]:] == 5.0).all())
    torch.testing.assert_close(out[:, :cu[-1]], want + 5.0 if accumulate else want, rtol=2.0 ** -18, atol=0)
