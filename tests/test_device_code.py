"""The built device code (no GPU), looked through for a form that faulted once: a register copy in front of the
instruction that gives a block its lanes back.  The copy then runs with the lanes of the branch that ended there, the
others keep what the register held before, and an address formed from it goes anywhere.  It came from loops whose lanes
left a row's end one by one, with masks spilled; the compiler says nothing."""
import os
import re
import shutil
import subprocess

import pytest

from retnet_retention_chunkwise_amd._lib import LIB_PATH

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
COPY = re.compile(r"v_(accvgpr_write|accvgpr_read|accvgpr_mov|mov)_b")
OTHER = re.compile(r"(s_(?!or_b64 exec)|v_writelane|v_readlane)")


def copies_before_lanes(lines):
    """(kernel, instruction) of copies that come first in a block, in front of its `s_or_b64 exec, exec, ...`."""
    kernel, found, ahead, first = None, [], [], True
    for line in lines:
        name = re.match(r"(?:[0-9a-f]+ )?<?(_Z\w+)>?:", line)
        text = line.strip()
        if name or re.match(r"(<L\d+>|\.?LBB\w+):", text):
            kernel = name.group(1) if name else kernel
            ahead, first = [], True
        elif not text or text[0] in ";." or not first:
            continue
        elif text.startswith("s_or_b64 exec, exec"):
            found += [(kernel, x) for x in ahead]
            first = False
        elif COPY.match(text):
            ahead.append(text)
        elif not OTHER.match(text) or text.startswith(("s_cbranch", "s_branch", "s_endpgm")):
            first = False
    return found


def test_the_form_is_recognised():
    bad = """_Zkernel:
    v_mov_b32_e32 v1, v2
    s_endpgm
.LBB7_132:
    v_readlane_b32 s0, v9, 3
    v_accvgpr_write_b32 a5, v19
    v_readlane_b32 s1, v9, 4
    s_or_b64 exec, exec, s[0:1]
    v_add_u32_e32 v1, v2, v3
""".splitlines()
    assert copies_before_lanes(bad) == [("_Zkernel", "v_accvgpr_write_b32 a5, v19")]
    good = [x for x in bad if "a5" not in x] + ["    v_accvgpr_write_b32 a5, v19"]
    assert copies_before_lanes(good) == []
    # behind another vector instruction the lanes are wanted as they are
    assert copies_before_lanes(bad[:4] + ["    v_add_u32_e32 v7, v8, v9"] + bad[4:]) == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_no_copy_before_a_block_has_its_lanes(tmp_path):
    lib = shutil.copy(LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", os.path.basename(lib)], cwd=tmp_path, check=True, stdout=subprocess.DEVNULL)
    parts = sorted(p for p in os.listdir(tmp_path) if p.endswith("gfx950"))
    blocks, kernels, found = 0, set(), []
    for p in parts:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", p], cwd=tmp_path, check=True,
                              stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True).stdout.splitlines()
        kernels |= {m.group(1) for m in (re.match(r"[0-9a-f]+ <(_Z\w+)>:", x) for x in text) if m}
        blocks += sum("s_or_b64 exec, exec" in x for x in text)
        found += copies_before_lanes(text)
    assert sum("attention" in k for k in kernels) >= 50 and blocks > 100, (len(kernels), blocks)
    assert not found, found
