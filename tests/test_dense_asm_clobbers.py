"""Assembly in the device sources names what it writes: without that the
compiler may keep a value of its own in the register."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_routed_expert_fp32_amd",
                    "csrc")


def blocks(text):
    """The argument text of every asm statement."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h"))),
                         ids=os.path.basename)
def test_m0_is_named_where_it_is_written(path):
    for b in blocks(open(path).read()):
        if re.search(r"s_mov_b32\s+m0\b", b):
            clobbers = b.rsplit(":", 1)[1] if b.count(":") >= 3 else ""
            assert '"m0"' in clobbers, b
