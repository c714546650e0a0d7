"""Assembly in the device sources names what it writes: without that the
compiler may keep a value of its own in the register."""
import glob
import os
import re
import shutil
import subprocess

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


def close_vector_writes(asm):
    """(loads with a scalar base, those of them whose base a vector instruction
    wrote less than five wait states before)."""
    code = [l.split(";")[0].strip() for l in asm.splitlines()]
    code = [l for l in code if l and (l.startswith((".LBB", "_Z")) or not l.startswith((".", "#")))]
    loads, close = 0, []
    for at, line in enumerate(code):
        m = re.match(r"global_load_lds_dwordx4 v\S+, s\[(\d+):(\d+)\]", line)
        if not m:
            continue
        loads += 1
        base, waits, k = {int(m[1]), int(m[2])}, 0, at - 1
        while waits < 5 and not code[k].startswith("_Z"):
            w = re.match(r"v_\S+ s(?:(\d+)\b|\[(\d+):(\d+)\])", code[k])
            if w and base & set(range(int(w[1] or w[2]), int(w[1] or w[3]) + 1)):
                close.append((line, code[k], waits))
            if not code[k].startswith(".LBB"):
                waits += int(code[k].split()[1]) + 1 if code[k].startswith("s_nop") else 1
            k -= 1
    return loads, close


def test_the_check_sees_a_close_write():
    asm = "_Zk:\nv_readfirstlane_b32 s9, v1\ns_mov_b32 m0, s4\ns_nop %d\nglobal_load_lds_dwordx4 v2, s[8:9]\n"
    assert close_vector_writes(asm % 0)[0] == 1 and len(close_vector_writes(asm % 0)[1]) == 1
    assert close_vector_writes(asm % 3) == (1, [])


def test_bases_of_loads_into_lds_are_scalar_results(tmp_path):
    hipcc = shutil.which("hipcc")
    if not hipcc:
        pytest.skip("no hipcc")
    from quantized_routed_expert_fp32_amd.csrc import build as B
    out = str(tmp_path / "dense.s")
    subprocess.run([hipcc, *B.HIPCC_FLAGS, "-S", "--cuda-device-only", os.path.join(CSRC, "dense.hip"), "-o", out],
                   check=True, capture_output=True, timeout=600)
    loads, close = close_vector_writes(open(out).read())
    assert loads > 100 and not close, close
