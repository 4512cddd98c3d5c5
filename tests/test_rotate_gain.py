"""The gain a Rotary takes where none is given.  Runs without a GPU."""
import math

import pytest

torch = pytest.importorskip("torch")

import compressed_index_matmul_amd as vq  # noqa: E402


@pytest.mark.parametrize("factor", [0.25, 1.0, 1.5, 16.0, 40.0])
def test_yarn(factor):
    """ln(f) / 10 + 1 of a longer context, none of a shorter one."""
    scaling = dict(kind="yarn", factor=factor, original=4096)
    want = 1.0 + math.log10(factor) / math.log10(math.e) / 10.0 if factor > 1.0 else 1.0
    assert vq.Rotary(64, scaling=scaling, device="cpu").gain == pytest.approx(want, rel=1e-12)
    r = vq.Rotary(64, scaling=dict(scaling, gain=0.7), device="cpu")
    assert r.gain == 0.7 and r.desc.gain == pytest.approx(0.7, rel=2.0 ** -24)


def test_others_have_none():
    for scaling in (None, dict(kind="linear", factor=4.0), dict(kind="base", factor=4.0),
                    dict(kind="bands", factor=4.0, original=4096)):
        assert vq.Rotary(64, scaling=scaling, device="cpu").gain == 1.0
