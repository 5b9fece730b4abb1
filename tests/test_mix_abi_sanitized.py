"""The lapmix ABI tests (tests/test_mix_abi.py) against the build of the library whose host
code runs under AddressSanitizer and UndefinedBehaviorSanitizer, as
tests/test_abi_sanitized.py does for the attention's."""

import os
import subprocess
import sys

from test_abi_sanitized import ROOT, _env


def test_mix_abi_under_sanitizers():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "not gpu", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_mix_abi.py")],
                       cwd=ROOT, env=_env(), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "passed" in r.stdout and "failed" not in r.stdout, r.stdout[-2000:]
