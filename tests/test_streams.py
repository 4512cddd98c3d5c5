"""Where the calls' own tensors come from when they are told a stream: from
that stream's memory, and what they return is kept for the caller's stream.
CPU tensors stand in for the GPU's, and recorders for the allocator, the
streams and the library."""
import contextlib

import pytest
import torch

import compressed_index_matmul_amd as vq

CURRENT, SIDE = 0x10, 0x20


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream.cuda_stream]


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class World:
    def __init__(self):
        self.under, self.made, self.launched = [CURRENT], [], []


@pytest.fixture
def world(monkeypatch):
    w = World()

    @contextlib.contextmanager
    def stream(st):
        w.under.append(st.cuda_stream)
        yield
        w.under.pop()

    real = torch.empty

    def empty(*shape, dtype=None, device=None):
        t = real(*shape, dtype=dtype).as_subclass(OnGpu)
        t.made_under = w.under[-1]
        w.made.append(t)
        return t

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(w.under[-1]))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(tuple(t.shape), dtype=t.dtype))
    from compressed_index_matmul_amd import attention
    for m in (attention, getattr(vq, "streams", None)):
        if m is not None:
            monkeypatch.setattr(m, "_raw_stream", lambda index: w.under[-1], raising=False)
    monkeypatch.setattr(attention, "_current_device", lambda: 0)

    def call(*args):
        w.launched.append(args[-1])
        return 0

    for name in attention.ATTN_EXPORTS:
        monkeypatch.setitem(attention._FN, name, (lambda *a: 64) if name.endswith("_size") else call)
    return w


def attention_calls():
    cache = vq.KV4Cache.from_buffers(on_gpu(2, 2, 2, 1024, dtype=torch.uint8), on_gpu(2, 2, 2, 8, 2, 8, dtype=torch.float16),
                                     on_gpu(2, 2, 32, dtype=torch.float32), on_gpu(2, 2, 32, dtype=torch.int32))
    q, k, cu = on_gpu(3, 4, 64), on_gpu(3, 2, 64), on_gpu(2, dtype=torch.int32)
    t, n, lse = on_gpu(1, 1, dtype=torch.int32), on_gpu(1, dtype=torch.int32), on_gpu(4, 3, dtype=torch.float32)
    return {
        "attn_prompt": lambda s: vq.attn_prompt(q, k, k, cu, return_lse=True, stream=s),
        "attn_prompt_weights": lambda s: vq.attn_prompt_weights(q, k, lse, cu, stream=s),
        "kv4_append": lambda s: vq.kv4_append(cache, k, k, cu, t, stream=s),
        "kv4_read": lambda s: vq.kv4_read(cache, cu, t, 3, stream=s),
        "kv4_attend": lambda s: vq.kv4_attend(q[:1], cache, t, n, return_lse=True, stream=s),
        "kv4_evict": lambda s: vq.kv4_evict(cache, t, n, n, keep=4, recent=1, stream=s),
    }


MADE = {"attn_prompt": 3, "attn_prompt_weights": 2, "kv4_append": 0, "kv4_read": 2, "kv4_attend": 3, "kv4_evict": 1}


@pytest.mark.parametrize("name", list(MADE))
@pytest.mark.parametrize("stream", [None, SIDE, CURRENT])
def test_attention_allocates_on_its_stream(world, name, stream):
    got = attention_calls()[name](stream)
    want = CURRENT if stream is None else stream
    returned = [] if got is None else list(got) if isinstance(got, tuple) else [got]
    assert world.launched == [want] and len(world.made) == MADE[name]
    assert [t.made_under for t in world.made] == [want] * MADE[name]
    for t in returned:
        recorded = [s for s in getattr(t, "recorded", []) if s != want]
        assert recorded == ([] if want == CURRENT else [CURRENT])


def product_calls():
    w = vq.VQWeight.__new__(vq.VQWeight)
    w.n_out, w.k_in, w.n_stages, w.device, w.desc = 16, 64, 1, torch.device("cuda", 0), vq.VQWeightDesc()
    x, signs = on_gpu(3, 64), on_gpu(64, dtype=torch.int8)
    return {
        "vq_unpack_dequant": lambda s: vq.vq_unpack_dequant(w, stream=s),
        "vq_gemv": lambda s: vq.vq_gemv(w, x, stream=s),
        "vq_gemm": lambda s: vq.vq_gemm(w, x, stream=s),
        "vq_gemm_noalloc": lambda s: vq.vq_gemm_noalloc(w, x, on_gpu(3, 16, dtype=torch.float32), stream=s),
        "rht_apply": lambda s: vq.rht_apply(x, signs, 64, stream=s),
        "rht_apply_shards": lambda s: vq.rht_apply_shards(x, signs, 64, [32, 32], stream=s),
        "vq_gemv_rht": lambda s: vq.vq_gemv_rht(w, x, signs, 64, stream=s),
    }


PRODUCTS = {"vq_unpack_dequant": 2, "vq_gemv": 1, "vq_gemm": 2, "vq_gemm_noalloc": 0, "rht_apply": 1,
            "rht_apply_shards": 1, "vq_gemv_rht": 1}


@pytest.mark.parametrize("name", list(PRODUCTS))
@pytest.mark.parametrize("stream", [None, SIDE, CURRENT])
def test_products_allocate_on_their_stream(world, monkeypatch, name, stream):
    class Library:
        def __getattr__(self, f):
            return (lambda *a: 64) if f.endswith("_size") else (lambda *a: world.launched.append(a[-1]) or 0)

    monkeypatch.setattr(vq, "lib", Library)
    world.made.clear()
    got = product_calls()[name](stream)
    want = CURRENT if stream is None else stream
    returned = [] if PRODUCTS[name] == 0 else list(got) if isinstance(got, tuple) else [got]
    assert world.launched == [want] and len(world.made) == PRODUCTS[name]
    assert [t.made_under for t in world.made] == [want] * PRODUCTS[name]
    for t in returned:
        recorded = [s for s in getattr(t, "recorded", []) if s != want]
        assert recorded == ([] if want == CURRENT else [CURRENT])


def test_arguments_that_are_no_tensors(world):
    q, k = on_gpu(3, 4, 64), on_gpu(3, 2, 64)
    for call in (lambda: vq.attn_prompt(q, k, k, [0, 3]), lambda: vq.attn_prompt_weights(q, k, on_gpu(4, 3), [0, 3]),
                 lambda: vq.attn_prompt(q, k, k, on_gpu(2, dtype=torch.int32), [0, 3]),
                 lambda: vq.attn_prompt(q, k, k, on_gpu(2, dtype=torch.int32), workspace=64),
                 lambda: vq.KV4Cache.from_buffers([1], [2], [3], [4])):
        with pytest.raises(TypeError):
            call()
