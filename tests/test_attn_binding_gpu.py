"""Refusals of the attention binding that need GPU tensors to be reached."""
import pytest
import torch

from attntest import ints
from vqtest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    ensure_built()
    import compressed_index_matmul_amd as m
    m.lib()
    return m


def x(n=4, h=2, d=64, dtype=torch.bfloat16):
    return torch.zeros((n, h, d), dtype=dtype, device="cuda")


def test_prompt_refusals(vq):
    cu = ints([0, 4])
    bad = [
        (TypeError, (x(dtype=torch.float32), x(), x(), cu)), (TypeError, (x(), x(dtype=torch.float16), x(), cu)),
        (ValueError, (x(), x(), x(dtype=torch.float16), cu)), (ValueError, (x(), x(5), x(5), cu)),
        (ValueError, (x(), x(), x(5), cu)), (ValueError, (x(h=3), x(), x(), cu)), (ValueError, (x(d=96), x(d=96), x(d=96), cu)),
        (ValueError, (x(), x(d=128), x(d=128), cu)), (ValueError, (x(), x(), x(), cu.long())),
        (ValueError, (x(), x(), x(), cu[None])), (ValueError, (x(), x(), x(), cu.cpu())),
        (ValueError, (x(d=128)[:, :, ::2], x(), x(), cu)), (ValueError, (x(), x()[:, :1].expand(-1, 2, -1), x(), cu)),
        (ValueError, (x(d=128)[:, :, 4:68], x(), x(), cu)), (ValueError, (x(), x(), x(), ints([0]))),
    ]
    for err, args in bad:
        with pytest.raises(err):
            vq.attn_prompt(*args)
    for kw in (dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(vq.VQError):
            vq.attn_prompt(x(), x(), x(), cu, **kw)
    with pytest.raises(ValueError):
        vq.attn_prompt(x(), x(), x(), cu, out=x(5))
    lse = torch.zeros((2, 4), device="cuda")
    for kw in (dict(last=-1), dict(accumulate=True), dict(out=torch.zeros((2, 5), device="cuda"))):
        with pytest.raises(ValueError):
            vq.attn_prompt_weights(x(), x(), lse, cu, **kw)
    with pytest.raises(ValueError):
        vq.attn_prompt_weights(x(), x(), lse.t(), cu)


def test_cache_refusals(vq):
    c = vq.KV4Cache(2, 32, 2, 64)
    t, n, cu = ints([[0]]), ints([1]), ints([0, 4])
    for err, args in [
            (ValueError, (x(h=3), x(h=3), cu, t)), (ValueError, (x(), x(5), cu, t)), (TypeError, (x(), x(dtype=torch.float16), cu, t)),
            (TypeError, (x(dtype=torch.int16), x(dtype=torch.int16), cu, t)), (ValueError, (x(), x(), ints([0, 2, 4]), t)),
            (ValueError, (x(), x(), cu, t.long())), (ValueError, (x(), x(), cu, t[0])), (ValueError, (x(), x(), cu, t, ints([1, 2])))]:
        with pytest.raises(err):
            vq.kv4_append(c, *args)
    with pytest.raises(ValueError):
        vq.kv4_append(c, x(), x(), cu, t, weights=torch.zeros((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        vq.kv4_read(c, cu, t, -1)
    with pytest.raises(TypeError):
        vq.kv4_read(c, cu, t, 4, dtype=torch.float64)
    for q, err in ((x(2), ValueError), (x(1, 3), ValueError), (x(1, d=128), ValueError), (x(1, dtype=torch.float32), TypeError)):
        with pytest.raises(err):
            vq.kv4_attend(q, c, t, n)
    for kw in (dict(max_len=-1), dict(out=x(2)), dict(workspace=torch.zeros(4))):
        with pytest.raises(ValueError):
            vq.kv4_attend(x(1), c, t, n, **kw)
    with pytest.raises(ValueError):
        vq.kv4_attend(x(1), c, t, None)
    for keep, recent in ((0, 0), (4, 5), (4, -1)):
        with pytest.raises(ValueError):
            vq.kv4_evict(c, t, n, n, keep, recent)
    with pytest.raises(ValueError):
        vq.kv4_evict(c, t, n, ints([1, 2]), 4, 2)
