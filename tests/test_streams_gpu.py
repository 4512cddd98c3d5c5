"""Calls told a stream: their results come from that stream's memory, also
where it is given as a raw handle, and equal those of the current stream."""
import numpy as np
import pytest

from attntest import heads, ints, new_cache, offsets
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


def pool_of(t):
    """The stream whose memory a tensor is in."""
    import torch
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("raw", [False, True])
def test_attention_on_a_stream(vq, raw):
    """Inputs made on the side stream, while the current stream frees and
    reuses blocks of the results' sizes."""
    import torch
    rng = np.random.default_rng(5)
    side = torch.cuda.Stream()
    n = 3000
    with torch.cuda.stream(side):
        cu, ck = ints([0, 40, 130]), ints([0, 100, n])
        q, _ = heads(rng, 130, 8, 128, "bf16")
        k, _ = heads(rng, n, 2, 128, "bf16")
        cache = new_cache(vq, 96, 64, 2, 128)
        t = torch.arange(96, dtype=torch.int32, device="cuda").view(2, 48)
        lens = ints([100, n - 100])
    side.synchronize()

    def run(stream):
        out, lse = vq.attn_prompt(q, k, k, cu, ck, return_lse=True, stream=stream)
        w = vq.attn_prompt_weights(q, k, lse, cu, ck, stream=stream)
        vq.kv4_append(cache, k, k, ck, t, weights=w, stream=stream)
        rk, rv = vq.kv4_read(cache, ck, t, n, stream=stream)
        o2, l2 = vq.kv4_attend(q[:2], cache, t, lens, add_weights=True, return_lse=True, stream=stream)
        vq.kv4_evict(cache, t, lens, lens, keep=500, recent=100, stream=stream)
        return [out, lse, w, rk, rv, o2, l2]

    with torch.cuda.stream(side):
        want = [x.clone() for x in run(None)]
        codes, weights = cache.codes.clone(), cache.weights.clone()
    side.synchronize()
    for _ in range(3):
        busy = [torch.empty_like(x) for x in want]
        for x in busy:
            x.fill_(7)
        del busy, x  # their blocks are free again for the current stream, which has yet to write them
        got = run(side.cuda_stream if raw else side)
        assert [pool_of(x) for x in got] == [side.cuda_stream] * len(got)
        torch.cuda.current_stream().wait_stream(side)
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
        assert torch.equal(cache.codes, codes) and torch.equal(cache.weights.view(torch.int32), weights.view(torch.int32))
        torch.cuda.synchronize()


def test_default_stream_by_its_handle(vq):
    """Handle 0 from within another stream."""
    import torch
    rng = np.random.default_rng(6)
    _, cu = offsets([40])
    q, _ = heads(rng, 40, 2, 64, "bf16")
    want = vq.attn_prompt(q, q, q, cu)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = vq.attn_prompt(q, q, q, cu, stream=0)
        assert pool_of(got) == torch.cuda.default_stream().cuda_stream
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_products_on_a_stream(vq):
    """The same for the products and transforms."""
    import torch
    import vqsynth
    from vqtest import device_weight
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        w = device_weight(vqsynth.random_weight(256, 512, 2, 12, 64, seed=3))
        x = torch.randn((100, 512), device="cuda").bfloat16()
        signs = (torch.randint(0, 2, (512,), device="cuda") * 2 - 1).to(torch.int8)
    side.synchronize()

    def run(stream):
        return [*vq.vq_unpack_dequant(w, stream=stream), vq.vq_gemv(w, x[:4], stream=stream), vq.vq_gemm(w, x, stream=stream),
                vq.rht_apply(x, signs, 512, stream=stream), vq.rht_apply_shards(x, signs, 256, [256, 256], stream=stream)]

    with torch.cuda.stream(side):
        want = run(None)
    side.synchronize()
    for stream in (side, side.cuda_stream):
        got = run(stream)
        assert [pool_of(t) for t in got] == [side.cuda_stream] * len(got)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
