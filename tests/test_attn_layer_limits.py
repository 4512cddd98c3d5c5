"""The example layer refuses budgets and prompts that its cache cannot hold,
whose last tokens the cache would drop."""
import os
import sys

import pytest

from vqtest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_budget_within_the_cache():
    import attention_layer
    for kw in (dict(keep=0), dict(keep=2048), dict(keep=300, max_len=256), dict(keep=64, max_len=40, page=64)):
        with pytest.raises(ValueError, match="keep"):
            attention_layer.AttentionLayer(2, **kw)


def test_prompt_within_the_cache():
    import attention_layer
    layer = attention_layer.AttentionLayer.__new__(attention_layer.AttentionLayer)
    layer.capacity = 128
    with pytest.raises(ValueError, match="prompt"):
        layer.prompt(None, [5, 129])
