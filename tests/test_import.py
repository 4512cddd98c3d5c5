"""Importing the package needs numpy only: torch comes with the first call
that handles its tensors."""
import subprocess
import sys

import compressed_index_matmul_amd as vq
from vqtest import ROOT, ensure_built


def test_import_and_library_without_torch():
    ensure_built()
    code = ("import sys\n"
            "sys.modules['torch'] = None  # importing it fails\n"
            "import compressed_index_matmul_amd as vq\n"
            "assert vq.vq_version() >= 6 and vq.VQ_F16 == 2 and 'attn_prompt' in dir(vq)\n"
            "assert vq.lib().attn_prompt.argtypes and vq.EXPORTS\n"
            "import compressed_index_matmul_amd.build\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr


def test_attention_names():
    from compressed_index_matmul_amd import attention
    assert set(attention.__all__) <= set(vq.__all__)
    for name in attention.__all__:
        assert getattr(vq, name) is getattr(attention, name)
    namespace = {}
    exec("from compressed_index_matmul_amd import *", namespace)
    assert all(name in namespace for name in vq.__all__)
    assert not hasattr(vq, "no_such_name")
