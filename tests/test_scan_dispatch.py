"""Which launches the scan takes a batch of prompts in (CPU; the launchers are stubs)."""
import os
import subprocess

import pytest

from tests.scan_dispatch_cases import CASES
from tests.test_sanitizers import HIPCC, ROOT


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("dispatch") / "dispatch")
    csrc = os.path.join(ROOT, "ssm_decode_amd", "csrc")
    r = subprocess.run([HIPCC, "-O1", "-std=c++17", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"),
                        os.path.join(csrc, "sk_api.cpp"), os.path.join(csrc, "sk_seq_api.cpp"),
                        os.path.join(ROOT, "tests", "sequence_dispatch_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


@pytest.mark.parametrize("name", sorted(CASES))
def test_launches(driver, name):
    H, G, dk, dv, act, lens, want = CASES[name]
    r = subprocess.run([driver] + [str(x) for x in (H, G, dk, dv, int(act == "f32"), sum(lens), len(lens))], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.splitlines() == want


def test_every_form_is_there():
    """Both launches with prompts on both sides of the border, and segments of every join."""
    said = [w for c in CASES.values() for w in c[6]]
    assert {"chunks 24 0", "step 24 0", "chunks -1 0", "step all 0", "chunks -1 128 launch", "chunks -1 256 each",
            "chunks -1 256 launch", "chunks -1 512 launch", "step all 32 launch"} <= set(said)
    for c in CASES.values():
        if c[6][0] == "chunks 24 0" and max(c[5]) > 5:
            assert {24, 25} <= set(c[5])
