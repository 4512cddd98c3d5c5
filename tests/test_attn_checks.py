"""The attention entry points refuse every invalid argument on the host,
before any HIP call: through the C ABI with stand-in addresses, and through
the Python binding.  They run without a GPU."""
import ctypes

import pytest
import torch

import compressed_index_matmul_amd as vq
from compressed_index_matmul_amd.attention import AttnBatch, AttnHeads, KV4CacheDesc, KV4Seqs
from vqtest import ensure_built

OK, NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, HIP, VALUE, WORKSPACE = 0, -1, -2, -3, -4, -5, -6, -7, -8
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    ensure_built()
    return vq.lib()


def batch(**kw):
    b = AttnBatch(1, 4, 2, 64, 3, 10, 12, 1, 0.125, 0, FAKE, FAKE)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def rows(data=FAKE, ts=256, hs=64):
    return AttnHeads(data, ts, hs)


BATCH_ERRORS = [
    (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(n_q_heads=0), SHAPE), (dict(n_kv_heads=0), SHAPE),
    (dict(n_q_heads=5), SHAPE), (dict(n_q_heads=65536), SHAPE), (dict(n_seqs=-1), SHAPE), (dict(total_q=-1), SHAPE),
    (dict(total_k=-1), SHAPE), (dict(reserved=1), SHAPE), (dict(causal=2), VALUE), (dict(scale=0.0), VALUE),
    (dict(scale=-1.0), VALUE), (dict(scale=float("nan")), VALUE), (dict(scale=float("inf")), VALUE),
    (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(cu_q=None), NULL), (dict(cu_k=None), NULL),
    (dict(cu_q=FAKE + 2), ALIGN), (dict(total_q=2**31 - 1, n_q_heads=64), SHAPE),
]
ROW_ERRORS = [(dict(data=None), NULL), (dict(data=FAKE + 8), ALIGN), (dict(ts=0), SHAPE), (dict(ts=-256), SHAPE),
              (dict(ts=100), SHAPE), (dict(hs=0), SHAPE), (dict(hs=4), SHAPE), (dict(ts=1 << 22), SHAPE),
              (dict(hs=1 << 40), SHAPE)]


@pytest.mark.parametrize("kw,want", BATCH_ERRORS)
def test_prompt_batch(L, kw, want):
    assert L.attn_prompt(batch(**kw), rows(), rows(), rows(), FAKE, None, FAKE, 1 << 40, None) == want
    if "total_q" not in kw or kw["total_q"] < 0:
        assert L.attn_prompt_weights(batch(**kw), rows(), rows(), FAKE, 0, 0, FAKE, FAKE, 1 << 40, None) == want


@pytest.mark.parametrize("kw,want", ROW_ERRORS)
def test_prompt_rows(L, kw, want):
    for i in range(3):
        h = [rows(), rows(), rows()]
        h[i] = rows(**kw)
        assert L.attn_prompt(batch(), *h, FAKE, None, FAKE, 1 << 40, None) == want
        if i < 2:
            assert L.attn_prompt_weights(batch(), *h[:2], FAKE, 0, 0, FAKE, FAKE, 1 << 40, None) == want


def prompt(L, b=None, q=None, out=FAKE, lse=None, ws=FAKE, n=1 << 40):
    return L.attn_prompt(b or batch(), q or rows(), rows(), rows(), out, lse, ws, n, None)


def gather(L, b=None, lse=FAKE, last=0, accumulate=0, out=FAKE, ws=FAKE, n=1 << 40):
    return L.attn_prompt_weights(b or batch(), rows(), rows(), lse, last, accumulate, out, ws, n, None)


def test_prompt_pointers(L):
    assert L.attn_prompt(None, rows(), rows(), rows(), FAKE, None, FAKE, 1 << 40, None) == NULL
    assert L.attn_prompt(batch(), None, rows(), rows(), FAKE, None, FAKE, 1 << 40, None) == NULL
    assert prompt(L, out=None) == NULL and prompt(L, ws=None) == NULL
    assert prompt(L, out=FAKE + 2) == ALIGN and prompt(L, lse=FAKE + 2) == ALIGN and prompt(L, ws=FAKE + 8) == ALIGN
    assert gather(L, lse=None) == NULL and gather(L, out=None) == NULL and gather(L, ws=None) == NULL
    assert gather(L, ws=FAKE + 8) == ALIGN and gather(L, last=-1) == SHAPE and gather(L, accumulate=2) == VALUE


def test_prompt_workspace(L):
    """Few rows against many keys need one; what is refused sizes to 0."""
    b = batch(total_q=100, total_k=5000, n_seqs=1)
    need = L.attn_prompt_workspace_size(b)
    assert need > 0 and prompt(L, b, n=need - 1) == WORKSPACE and prompt(L, b, ws=None, n=0) == WORKSPACE
    assert L.attn_prompt_workspace_size(batch(total_q=100000, total_k=100000)) == 0
    assert L.attn_prompt_workspace_size(batch(total_q=100, total_k=5000, cu_q=None, cu_k=None, n_seqs=1)) == need
    assert L.attn_prompt_workspace_size(batch(head_dim=80)) == 0 and L.attn_prompt_workspace_size(None) == 0
    b = batch(total_q=5000, total_k=100, n_seqs=1)
    need = L.attn_prompt_weights_workspace_size(b, 0)
    assert need > 0 and gather(L, b, n=need - 1) == WORKSPACE
    assert L.attn_prompt_weights_workspace_size(b, -1) == 0
    assert L.attn_prompt_weights_workspace_size(batch(total_q=5000, total_k=10**6), 0) == 0


def test_nothing_to_do_touches_no_device(L):
    assert L.attn_prompt(batch(total_q=0), rows(None), rows(), rows(), None, None, None, 0, None) == OK
    assert L.attn_prompt_weights(batch(total_k=0), rows(), rows(None), FAKE, 0, 0, None, None, 0, None) == OK
    assert L.kv4_append(cache(), seqs(), rows(), rows(), 1, 0, FAKE, None, None, None) == OK
    assert L.kv4_read(cache(), seqs(), FAKE, 0, 1, None, None, None) == OK
    assert L.kv4_attend(cache(), seqs(n_seqs=0), rows(), 1, 4, 1.0, 64, 0, None, None, None, 0, None) == OK
    assert L.kv4_evict(cache(), seqs(), FAKE, 64, 0, 64, None, 0, None) == OK  # nothing can be longer than keep


def cache(**kw):
    c = KV4CacheDesc(10, 32, 2, 64, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seqs(**kw):
    s = KV4Seqs(3, 4, FAKE, FAKE)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


CACHE_ERRORS = [(dict(n_pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=48), SHAPE),
                (dict(page_size=1056), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(head_dim=96), UNSUPPORTED),
                (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(weights=None), NULL), (dict(pos=None), NULL),
                (dict(codes=FAKE + 8), ALIGN), (dict(scales=FAKE + 4), ALIGN), (dict(weights=FAKE + 4), ALIGN),
                (dict(pos=FAKE + 4), ALIGN)]
SEQ_ERRORS = [(dict(n_seqs=-1), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=2**26), SHAPE),
              (dict(block_table=None), NULL), (dict(block_table=FAKE + 2), ALIGN), (dict(lens=FAKE + 1), ALIGN)]


def each_kv4(L, c, s):
    yield L.kv4_append(c, s, rows(), rows(), 1, 5, FAKE, None, None, None)
    yield L.kv4_read(c, s, FAKE, 5, 1, FAKE, FAKE, None)
    yield L.kv4_attend(c, s, rows(), 1, 4, 1.0, 64, 0, FAKE, None, FAKE, 1 << 30, None)
    yield L.kv4_evict(c, s, FAKE, 16, 0, 64, FAKE, 1 << 30, None)


@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_cache_descriptor(L, kw, want):
    assert list(each_kv4(L, cache(**kw), seqs())) == [want] * 4
    assert list(each_kv4(L, None, seqs())) == [NULL] * 4
    if want in (SHAPE, UNSUPPORTED):
        assert L.kv4_attend_workspace_size(cache(**kw), 3, 4, 64, 1) == 0
        assert L.kv4_evict_workspace_size(cache(**kw), 3, 16, 64) == 0


@pytest.mark.parametrize("kw,want", SEQ_ERRORS)
def test_sequences(L, kw, want):
    assert list(each_kv4(L, cache(), seqs(**kw))) == [want] * 4
    assert list(each_kv4(L, cache(), None)) == [NULL] * 4


@pytest.mark.parametrize("kw,want", ROW_ERRORS)
def test_cache_rows(L, kw, want):
    assert L.kv4_append(cache(), seqs(), rows(**kw), rows(), 1, 5, FAKE, None, None, None) == want
    assert L.kv4_append(cache(), seqs(), rows(), rows(**kw), 1, 5, FAKE, None, None, None) == want
    assert L.kv4_attend(cache(), seqs(), rows(**kw), 1, 4, 1.0, 64, 0, FAKE, None, FAKE, 1 << 30, None) == want


def test_append_and_read_arguments(L):
    def append(dtype=1, total=5, cu=FAKE, pos=None, weights=None):
        return L.kv4_append(cache(), seqs(), rows(), rows(), dtype, total, cu, pos, weights, None)

    assert append(dtype=3) == DTYPE and append(total=-1) == SHAPE and append(cu=None) == NULL
    assert append(cu=FAKE + 2) == ALIGN and append(pos=FAKE + 2) == ALIGN and append(weights=FAKE + 1) == ALIGN
    assert L.kv4_read(cache(), seqs(), FAKE, 5, 7, FAKE, FAKE, None) == DTYPE
    assert L.kv4_read(cache(), seqs(), FAKE, 5, 1, None, FAKE, None) == NULL
    assert L.kv4_read(cache(), seqs(), FAKE, 5, 1, FAKE, None, None) == NULL
    assert L.kv4_read(cache(), seqs(), FAKE, 5, 1, FAKE + 8, FAKE, None) == ALIGN
    assert L.kv4_read(cache(), seqs(), FAKE, -5, 1, FAKE, FAKE, None) == SHAPE


def test_attend_arguments(L):
    def attend(dtype=1, hq=4, scale=1.0, max_len=4000, weigh=0, out=FAKE, lse=None, ws=FAKE, n=1 << 30, s=None):
        return L.kv4_attend(cache(), s or seqs(), rows(), dtype, hq, scale, max_len, weigh, out, lse, ws, n, None)

    assert attend(dtype=0) == DTYPE and attend(hq=0) == SHAPE and attend(hq=3) == SHAPE and attend(max_len=-1) == SHAPE
    assert attend(hq=65536) == SHAPE and attend(scale=0.0) == VALUE and attend(scale=float("nan")) == VALUE
    assert attend(weigh=2) == VALUE and attend(out=None) == NULL and attend(ws=None) == NULL
    assert attend(out=FAKE + 4) == ALIGN and attend(lse=FAKE + 2) == ALIGN and attend(ws=FAKE + 8) == ALIGN
    assert attend(s=seqs(lens=None)) == NULL
    need = L.kv4_attend_workspace_size(cache(), 3, 4, 4000, 0)
    more = L.kv4_attend_workspace_size(cache(), 3, 4, 4000, 1)
    assert 0 < need < more
    assert attend(n=need - 1) == WORKSPACE and attend(n=need, weigh=1) == WORKSPACE and attend(ws=None, n=0) == WORKSPACE
    assert L.kv4_attend_workspace_size(cache(), 3, 3, 4000, 0) == 0 and L.kv4_attend_workspace_size(cache(), 0, 4, 40, 0) == 0


def test_evict_arguments(L):
    def evict(nxt=FAKE, keep=16, recent=4, max_len=64, ws=FAKE, n=1 << 30, s=None):
        return L.kv4_evict(cache(), s or seqs(), nxt, keep, recent, max_len, ws, n, None)

    assert evict(nxt=None) == NULL and evict(keep=0) == SHAPE and evict(recent=-1) == VALUE and evict(recent=17) == VALUE
    assert evict(max_len=-1) == SHAPE and evict(ws=None) == NULL and evict(nxt=FAKE + 2) == ALIGN
    assert evict(ws=FAKE + 8) == ALIGN and evict(s=seqs(lens=None)) == NULL
    need = L.kv4_evict_workspace_size(cache(), 3, 16, 64)
    assert need > 0 and evict(n=need - 1) == WORKSPACE
    assert L.kv4_evict_workspace_size(cache(), 3, 64, 64) == 0


def test_products_refuse_fp16(L):
    assert L.rht_apply(FAKE, vq.VQ_F16, 1, 64, FAKE, 64, FAKE, None) == DTYPE


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def host(n=4, h=2, d=64, dtype=torch.bfloat16):
    return torch.zeros((n, h, d), dtype=dtype)


@pytest.mark.parametrize("q,err", [
    (torch.zeros((4, 128), dtype=torch.bfloat16), ValueError),  # not [tokens, heads, channels]
    (host(), ValueError),                                       # host memory
    ([1, 2], TypeError),
])
def test_prompt_tensors(q, err):
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(err):
        vq.attn_prompt(q, host(), host(), cu)
    with pytest.raises(err):
        vq.attn_prompt_weights(q, host(), torch.zeros((2, 4)), cu)


@pytest.mark.parametrize("args", [dict(n_pages=0), dict(page_size=40), dict(page_size=16), dict(page_size=2048),
                                  dict(head_dim=96), dict(n_kv_heads=0)])
def test_cache_sizes(args):
    kw = dict(n_pages=2, page_size=32, n_kv_heads=2, head_dim=64, device="cpu")
    vq.KV4Cache(**kw)
    kw.update(args)
    with pytest.raises(ValueError):
        vq.KV4Cache(**kw)


def test_cache_buffers():
    c = vq.KV4Cache(2, 32, 3, 128, device="cpu")
    again = vq.KV4Cache.from_buffers(c.codes, c.scales, c.weights, c.pos)
    assert (again.n_pages, again.page_size, again.n_kv_heads, again.head_dim) == (2, 32, 3, 128)
    assert again.nbytes() == 2 * 3 * 32 * (2 * (64 + 16) + 8)
    for bad in ((c.codes[:, :, :, 1:], c.scales, c.weights, c.pos), (c.codes, c.scales.float(), c.weights, c.pos),
                (c.codes, c.scales, c.weights, c.pos.long()), (c.codes, c.scales, c.weights[:1], c.pos),
                (c.codes, c.scales, c.weights.transpose(0, 1).contiguous().transpose(0, 1), c.pos)):
        with pytest.raises(ValueError):
            vq.KV4Cache.from_buffers(*bad)


def test_host_cache_is_refused():
    c = vq.KV4Cache(2, 32, 2, 64, device="cpu")
    t, n = torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    for call in (lambda: vq.kv4_append(c, host(1), host(1), cu, t), lambda: vq.kv4_read(c, cu, t, 1),
                 lambda: vq.kv4_attend(host(1), c, t, n), lambda: vq.kv4_evict(c, t, n, n, 1, 0)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_descriptors_match_the_header():
    """Sizes of the mirrored structures, as the C compiler lays them out."""
    assert ctypes.sizeof(AttnHeads) == 24 and ctypes.sizeof(AttnBatch) == 56
    assert ctypes.sizeof(KV4CacheDesc) == 48 and ctypes.sizeof(KV4Seqs) == 24
