"""The host code of the scan, convolution, beam and reorder calls (sk_seq_api.cpp)
under AddressSanitizer and UndefinedBehaviorSanitizer, driven by
tests/sequence_validation_driver.cpp, and the slots that its plan gives to
random lists of prompts (CPU)."""
import os
import subprocess

import pytest

from tests.test_sanitizers import ENV_SAN, HIPCC, ROOT, SAN


def test_sequence_validation_under_sanitizers(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "sequence_san")
    flags = []
    for f in SAN:                       # host code only: each sanitizer flag after -Xarch_host
        flags += ["-Xarch_host", f]
    csrc = os.path.join(ROOT, "ssm_decode_amd", "csrc")
    cmd = [HIPCC, "-O1", "-g", "-std=c++17", "--offload-arch=gfx950"] + flags + \
          ["-I", os.path.join(ROOT, "include"), os.path.join(csrc, "sk_api.cpp"),
           os.path.join(csrc, "sk_seq_api.cpp"), os.path.join(ROOT, "tests", "sequence_validation_driver.cpp"),
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, env={**os.environ, **ENV_SAN}, timeout=120)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-3000:]
    assert "all checks passed" in out
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-3000:]
