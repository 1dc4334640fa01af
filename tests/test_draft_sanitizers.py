"""The host code of rotary positions and drafted tokens (argument checks, plans, workspace sizes) under
AddressSanitizer and UndefinedBehaviorSanitizer, as test_kv_sanitizers.py does for the cache.  No GPU is used."""
import os
import subprocess
import sys

import pytest

from block_wise_mixed_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.timeout(900)
def test_draft_host_suite_clean_under_sanitizers(tmp_path):
    rt = build.asan_runtime()
    if rt is None:
        pytest.skip("clang's shared ASan runtime is not installed")
    lib = str(tmp_path / "libmsq_asan.so")
    build.build_host_sanitized(lib)
    env = dict(os.environ)
    env.update({"LD_PRELOAD": rt, "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1:abort_on_error=0",
                "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1", "PYTHONMALLOC": "malloc", "MSQ_LIBRARY": lib})
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_draft_host.py"),
                        "-k", "not binding_refuses"],  # torch is not loaded under the runtime
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=800)
    log = r.stdout + r.stderr
    assert "Sanitizer" not in log and "runtime error" not in log, log[-4000:]
    assert r.returncode == 0, log[-4000:]
    assert " passed" in r.stdout
