"""A workspace of kv4_attend_chunk's size for the largest call of a program
serves its smaller ones.  Without a GPU an accepted call ends at its launch."""
import random

import numpy as np
import pytest

import compressed_index_matmul_amd as vq
from test_attn_checks import HIP, WORKSPACE, cache, seqs
from test_chunk_checks import chunk
from vqtest import ensure_built

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    ensure_built()
    if torch.cuda.is_available():
        pytest.skip("the accepted sizes would be launched on stand-in addresses")
    return vq.lib()


def size(L, c, hq, n, tq, max_len, max_q, window, sinks):
    return L.kv4_attend_chunk_workspace_size(c, n, hq, tq, window, sinks, max_len, max_q)


def call(L, c, hq, n, tq, max_len, max_q, window, sinks, ws):
    return chunk(L, c, seqs(n_seqs=n, max_pages=1 << 20), hq=hq, tq=tq, max_len=max_len, max_q=max_q, window=window, sinks=sinks,
                 n=ws)


def test_one_long_prompt_in_pieces(L):
    """The whole of it at once takes row tiles whole, its pieces are cut."""
    c = cache(n_kv_heads=8, head_dim=128)
    most = size(L, c, 32, 1, 4096, 16384, 4096, 0, 0)
    for tq in (4000, 2048, 1024, 300, 17, 1):
        assert size(L, c, 32, 1, tq, 16384, tq, 0, 0) <= most
        assert call(L, c, 32, 1, tq, 16384, tq, 0, 0, most) == HIP


@pytest.mark.parametrize("hkv,hq", [(1, 1), (3, 9), (8, 32), (8, 64), (4, 4), (1, 128), (64, 64)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_smaller_calls(L, d, hq, hkv):
    c, rng = cache(n_kv_heads=hkv, head_dim=d), random.Random(d + hq)

    def spread(top):
        return int(round(2.0 ** rng.uniform(0.0, np.log2(top))))

    for _ in range(150):
        n, tq, max_len = spread(300), spread(20000), spread(70000)
        max_q = rng.choice([tq, spread(tq), spread(64)])
        window, sinks = rng.choice([(0, 0), (0, 0), (spread(8000), rng.choice([0, 4, 100]))])
        most = size(L, c, hq, n, tq, max_len, max_q, window, sinks)
        assert call(L, c, hq, n, tq, max_len, max_q, window, sinks, most) == HIP
        for _ in range(6):
            less = [rng.choice([v, spread(v)]) for v in (n, tq, max_len, max_q)]
            assert size(L, c, hq, *less, window, sinks) <= most, (n, tq, max_len, max_q, less, window, sinks)
            assert call(L, c, hq, *less, window, sinks, most) == HIP, (n, tq, max_len, max_q, less, window, sinks)


def test_nothing_to_do_needs_nothing(L):
    c = cache(n_kv_heads=2, head_dim=64)
    assert size(L, c, 4, 3, 0, 20000, 0, 0, 0) == 0
    assert size(L, c, 4, 3, 5, 100, 5, 0, 0) == 0  # every row tile whole
    assert call(L, c, 4, 3, 200, 20000, 200, 0, 0, 0) == WORKSPACE
