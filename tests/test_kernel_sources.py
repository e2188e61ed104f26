"""What the kernel sources have to say to the compiler (read as text)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ssm_decode_amd", "csrc")


def _asm_statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*")) + glob.glob(os.path.join(CSRC, "*.inc"))):
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", open(path).read(), re.S):
            yield os.path.basename(path), m.group(1)


def test_assembly_that_sets_m0_says_so():
    """Otherwise the compiler may keep a value of its own in m0 across it."""
    setting = [(f, s) for f, s in _asm_statements() if re.search(r"s_mov_b32\s+m0", s)]
    assert len(setting) == 2               # copy16, copy16x4
    for f, s in setting:
        assert re.search(r'"m0"', s.rsplit(":", 1)[1]), (f, s)
