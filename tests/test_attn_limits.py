"""Sizes that no launch takes (2^32 work items) are refused by the checks, and
those just below are not: without a GPU an accepted call ends at its launch."""
import pytest

from test_attn_checks import FAKE, HIP, OK, SHAPE, batch, cache, rows, seqs
import compressed_index_matmul_amd as vq
from vqtest import ensure_built

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    ensure_built()
    if torch.cuda.is_available():
        pytest.skip("the accepted sizes would be launched on stand-in addresses")
    return vq.lib()


BIG = 1 << 62


def test_prompt(L):
    # 64 heads: 2^18 row blocks are one too many, with a sequence's spare one
    for tq, want in (((1 << 25) - 128 * 2, HIP), ((1 << 25) - 128, SHAPE), ((1 << 30), SHAPE)):
        b = batch(n_q_heads=64, n_kv_heads=64, n_seqs=1, total_q=tq, total_k=tq)
        assert L.attn_prompt(b, rows(), rows(), rows(), FAKE, None, FAKE, BIG, None) == want, tq
        assert L.attn_prompt_weights(b, rows(), rows(), FAKE, 0, 0, FAKE, FAKE, BIG, None) == want, tq


def test_gathered_weights_keep_their_pieces_within_a_launch(L):
    b = batch(n_q_heads=64, n_kv_heads=64, n_seqs=1, total_q=1 << 24, total_k=1 << 24)
    need = L.attn_prompt_weights_workspace_size(b, 0)
    assert need // (64 * (1 << 24) * 4) * (((1 << 24) // 128 + 1) * 64) < 1 << 24


def test_cache_calls(L):
    c = cache(n_kv_heads=32, head_dim=256)  # 8 workgroups a quad of slots
    for total, want in ((4 * ((1 << 21) - 7), HIP), (4 * ((1 << 21) - 6), SHAPE), (1 << 30, SHAPE)):
        assert L.kv4_append(c, seqs(), rows(), rows(), 1, total, FAKE, None, None, None) == want, total
        assert L.kv4_read(c, seqs(), FAKE, total, 1, FAKE, FAKE, None) == want, total


def test_attend(L):
    c = cache(n_pages=1 << 16, n_kv_heads=8, head_dim=128)
    s = seqs(n_seqs=4096, max_pages=1 << 18)

    def attend(max_len, weigh):
        return L.kv4_attend(c, s, rows(), 1, 32, 1.0, max_len, weigh, FAKE, None, FAKE, BIG, None)

    assert attend(1 << 20, 0) == HIP  # only the join of added weights grows with the lengths
    assert attend(1 << 20, 1) == SHAPE and L.kv4_attend_workspace_size(c, 4096, 32, 1 << 20, 1) == 0
    assert attend(500 * 1024, 1) == HIP
    c.n_pages = 1 << 10
    assert attend(1 << 20, 1) == HIP  # and no further than the pool


def test_evict(L):
    c = cache(n_kv_heads=32)

    def evict(n, keep, max_len):
        return L.kv4_evict(c, seqs(n_seqs=n, max_pages=1 << 18), FAKE, keep, 0, max_len, FAKE, BIG, None)

    assert evict(512, 1 << 16, 1 << 17) == HIP  # moves are taken in as many rounds as it needs
    assert evict((1 << 17) - 1, 16, 64) == HIP and evict(1 << 17, 16, 64) == SHAPE
    assert L.kv4_evict(c, seqs(), FAKE, 64, 0, 64, None, 0, None) == OK


def test_evict_workspace_holds_what_is_used():
    """Rows of up to 32768 slots keep their keys in registers."""
    ensure_built()
    size = vq.lib().kv4_evict_workspace_size
    for n, keep, max_len in ((64, 1024, 32768), (64, 1024, 32769), (3, 5000, 8191), (1, 1, 2)):
        r, moves = n * 2, min(keep, max_len - keep)
        most = r * (8 * moves + 4 + (4 * max_len if max_len > 32768 else 0))
        assert most <= size(cache(), n, keep, max_len) <= most + 3 * 256


def test_attend_workspace_grows_with_the_pool():
    """Scores are kept for slots that the pool can hold, not for every
    sequence at its bound."""
    ensure_built()
    size = vq.lib().kv4_attend_workspace_size
    c = cache(n_pages=200, page_size=64, n_kv_heads=8, head_dim=128)
    plain = size(c, 64, 64, 131072, 0)
    scores = size(c, 64, 64, 131072, 1) - plain
    assert 200 * 64 * 64 * 4 <= scores <= 200 * 64 * 64 * 4 + 64 * 64 * 8 + 512
    # and no more than the bound where that is less
    assert size(c, 2, 64, 100, 1) - plain <= 2 * 128 * 64 * 4 + 2 * 64 * 8 + 512
