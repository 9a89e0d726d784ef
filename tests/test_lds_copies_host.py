"""The copies into LDS in the built library's own gfx950 code: their LDS
address is M0, and a scalar write of M0 needs one wait state before a load
that reads it.  The compiler counts wait states between its own instructions
but not inside an inline-assembly string, so the string has to hold it."""
import glob
import os
import re
import shutil
import subprocess

import pytest

import int8_gemm_linear_amd as q

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def copies_without_wait(text):
    """(copies into LDS, those whose instruction before wrote M0) of a listing."""
    copies, bad, before = 0, 0, ""
    for line in text.splitlines():
        t = line.split("//")[0].strip()
        if not t:
            continue
        if re.match(r"(global_load|buffer_load|scratch_load)\S*", t) and re.search(r"load_lds|\blds\b", t):
            copies += 1
            bad += bool(re.match(r"s_\w+ m0\b", before))
        before = t
    return copies, bad


def test_the_search_sees_both_forms():
    near = "\ts_mov_b32 m0, s3 // 01\n\tglobal_load_lds_dwordx4 v2, s[4:5] // 02\n"
    apart = near.replace("\tglobal", "\ts_nop 0\n\tglobal")
    assert copies_without_wait(near) == (1, 1) and copies_without_wait(apart) == (1, 0)


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_m0_is_set_a_wait_state_before_every_copy(tmp_path):
    lib = shutil.copy(q.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, stdout=subprocess.DEVNULL)
    objects = glob.glob(str(tmp_path / "*gfx950"))
    assert objects
    copies = bad = 0
    for obj in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", obj], check=True, capture_output=True,
                              text=True).stdout
        c, b = copies_without_wait(text)
        copies, bad = copies + c, bad + b
    assert copies > 0 and bad == 0, f"{bad} of {copies} copies into LDS right behind a write of M0"
