"""The refusals of the attention, bias and dropout calls against the build of the library whose host code carries
AddressSanitizer and UndefinedBehaviorSanitizer, every finding fatal.  CPU only: that build launches no kernel."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_refusals_under_asan_and_ubsan():
    # imported here: the build script is host tooling that GPU runs do not carry
    from equivariant_gnn_electronic_amd import build_sanitized as bs
    lib = bs.build_if_stale()
    env = dict(os.environ, EGNN_LIBRARY=lib, LD_PRELOAD=bs.asan_runtime(), PYTHONMALLOC="malloc",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_attention_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert "passed" in r.stdout.strip().splitlines()[-1]
