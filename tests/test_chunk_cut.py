"""When kv4_attend_chunk cuts its work into shares: seen by the workspace that a
call asks for (without a GPU an accepted call ends at its launch)."""
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


def whole(L, d, hkv, hq, lq, most, max_q=None, window=0, sinks=0):
    """Whether row tiles of many rows are whole: then the call asks for the
    few-row kernel's area at most."""
    c, n = cache(n_kv_heads=hkv, head_dim=d), len(lq)
    few = 256 * (3 if d == 64 else 2) * 2 * 32 * (d * 4 + 8) + 256 * (1 + (n + 1) * 4 // 256)
    got = chunk(L, c, seqs(n_seqs=n, max_pages=1 << 20), hq=hq, tq=sum(lq), max_len=most, max_q=max_q or max(lq), window=window,
                sinks=sinks, n=few)
    assert got in (HIP, WORKSPACE)
    return got == HIP


@pytest.mark.parametrize("d,hkv,hq", [(64, 16, 64), (128, 8, 32), (256, 8, 32)])
@pytest.mark.parametrize("order", [1, -1])
def test_a_long_sequence_beside_short_ones_is_cut(L, d, hkv, hq, order):
    """Whole, its few row tiles would walk tens of thousands of slots on a handful
    of CUs long after the others have ended."""
    assert not whole(L, d, hkv, hq, [1200, 1200, 1200, 1200, 30][::order], 60030)
    assert not whole(L, d, hkv, hq, [1200] * 4 + [300], 40300)
    assert not whole(L, d, hkv, hq, [512] * 16 + [100], 30000)


@pytest.mark.parametrize("d,hkv,hq", [(64, 16, 64), (128, 8, 32), (256, 8, 32)])
def test_chunks_of_their_own_tokens_are_whole(L, d, hkv, hq):
    assert whole(L, d, hkv, hq, [4096], 4096)
    assert whole(L, d, hkv, hq, [2000] * 3, 4000)
    assert whole(L, d, hkv, hq, [4096] + [1] * 40, 4096)  # a prompt beside single tokens no longer than it
    assert whole(L, d, hkv, hq, [4096], 60000, window=1024, sinks=4)  # no row tile meets more than the window


def test_few_slots_are_whole_and_few_row_tiles_are_not(L):
    assert whole(L, 128, 8, 32, [100, 200], 500) and whole(L, 128, 8, 32, [300] * 8, 1000)
    assert not whole(L, 128, 8, 32, [1000], 2000)
