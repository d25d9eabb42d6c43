"""test_abi_rows.py on the build whose host code carries AddressSanitizer and
UndefinedBehaviorSanitizer, as test_abi_sanitized.py does with test_abi.py."""

import os
import subprocess
import sys

from decode_nvfp4_rtn_amd import build as qb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_abi_rows_under_host_sanitizers():
    lib = qb.build_sanitized(verbose=False)
    rt = qb.sanitizer_runtime()
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:verify_asan_link_order=0"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    env["QLIN_ABI_LIB"] = lib
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_rows.py")],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert " passed" in r.stdout and "AddressSanitizer" not in r.stderr
