"""The limits of the attention entry points under AddressSanitizer and
UndefinedBehaviorSanitizer: sizes near the ends of their types go through the
checks and plans of the host-sanitized build (host code only)."""
import subprocess
import sys

import pytest

from vqtest import ROOT


def test_limits_under_host_sanitizers():
    from compressed_index_matmul_amd import build
    try:
        build.asan_runtime()
    except (RuntimeError, OSError) as e:
        pytest.skip(f"no ASan runtime: {e}")
    build.build_hostsan()
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_attn_limits.py", "tests/test_streams.py"],
                       cwd=ROOT, env=build.hostsan_env(), capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
