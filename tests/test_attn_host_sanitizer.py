"""The attention entry points' argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer: the CPU checks again in a fresh Python on the
host-sanitized build (host code only)."""
import subprocess
import sys

import pytest

from vqtest import ROOT


@pytest.fixture(scope="module")
def hostsan_lib():
    from compressed_index_matmul_amd import build
    try:
        build.asan_runtime()
    except (RuntimeError, OSError) as e:
        pytest.skip(f"no ASan runtime: {e}")
    return build.build_hostsan()


def test_attn_checks_under_host_sanitizers(hostsan_lib):
    from compressed_index_matmul_amd import build
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_attn_checks.py"],
                       cwd=ROOT, env=build.hostsan_env(), capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
