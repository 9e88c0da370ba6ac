"""The built kernels' listing keeps the waits that an LDS copy
(global_load_lds_*) needs.  The copies are written in inline assembly, where
the compiler adds none:
  * one wait state after a scalar instruction has written M0, which holds the
    copy's LDS address (an s_nop or any other instruction between them);
  * five after a vector instruction (v_readlane, v_readfirstlane, a compare)
    has written a scalar register that the copy takes its base from.
CPU only: it reads the disassembly of the library that was built here."""
import os
import re
import struct
import subprocess

import pytest

import tiled_dense_gemm_loop_amd.build as b

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def device_images(path):
    """The gfx950 code objects in a library: one bundle per translation unit."""
    with open(path, "rb") as f:
        data = f.read()
    at = data.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, id_len = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + id_len] and size:
                yield data[at + offset:at + offset + size]
            p += 24 + id_len
        at = data.find(MAGIC, at + 1)


def scalars(text):
    """Numbers of the scalar registers that an operand text names."""
    regs = set()
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        regs.update(range(int(lo), int(hi) + 1))
    regs.update(int(n) for n in re.findall(r"\bs(\d+)\b", text))
    if "vcc" in text:
        regs.add(-1)
    return regs


def missing_waits(lines):
    """(kernel, earlier instruction, copy) wherever a wait is missing, and the
    number of copies."""
    bad, copies, name, before = [], 0, "", []
    for line in lines:
        m = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if m:
            name, before = m.group(1), []
            continue
        ins = line.split("//")[0].strip()
        if not line.startswith("\t") or not ins:
            continue
        op, _, operands = ins.partition(" ")
        if op.startswith("global_load_lds"):
            copies += 1
            base, states = scalars(operands), 0
            for prev_op, prev in reversed(before):
                dest = prev.split(",")[0]
                if states < 1 and prev_op.startswith("s_") and re.search(r"\bm0\b", dest):
                    bad.append((name, prev_op + " " + prev, ins))
                if prev_op.startswith("v_") and scalars(dest) & base:
                    bad.append((name, prev_op + " " + prev, ins))
                if prev_op.startswith("s_") and not prev_op.startswith(("s_nop", "s_cmp", "s_bitcmp")):
                    base -= scalars(dest)  # written since, by a scalar instruction
                states += int(prev, 0) + 1 if prev_op == "s_nop" else 1
                if states >= 5:
                    break
        before.append((op, operands.strip()))
        del before[:-6]
    return bad, copies


@pytest.mark.parametrize("text,faults", [
    ("s_mov_b32 m0, s4|global_load_lds_dwordx4 v1, s[2:3]", 1),
    ("s_add_i32 m0, s4, 64|global_load_lds_dwordx4 v[2:3], off", 1),
    ("s_mov_b32 m0, s4|s_nop 0|global_load_lds_dwordx4 v1, s[2:3]", 0),
    ("s_mov_b32 m0, s4|v_mov_b32 v1, v2|global_load_lds_dword v[2:3], off", 0),
    ("v_readlane_b32 s3, v9, 1|s_nop 3|global_load_lds_dwordx4 v1, s[2:3]", 1),
    ("v_readlane_b32 s3, v9, 1|s_nop 4|global_load_lds_dwordx4 v1, s[2:3]", 0),
    ("v_readfirstlane_b32 s8, v9|s_mov_b64 s[2:3], s[8:9]|global_load_lds_dwordx4 v1, s[2:3]", 0),
    ("v_cmp_gt_u32_e64 s[2:3], v1, v2|global_load_lds_dwordx4 v1, s[2:3]", 1),
])
def test_the_scan_itself(text, faults):
    bad, copies = missing_waits(["0000000000001000 <k>:"] + ["\t%s  // 0: 0" % i for i in text.split("|")])
    assert copies == 1 and len(bad) == faults


def test_every_copy_has_its_waits(tmp_path):
    if not os.path.exists(b.LIB_PATH):
        pytest.skip("build the library first (__graft_entry__.build())")
    copies = 0
    for i, image in enumerate(device_images(b.LIB_PATH)):
        path = tmp_path / ("image%d" % i)
        path.write_bytes(image)
        res = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, timeout=300)
        assert res.returncode == 0, res.stderr[-2000:]
        bad, n = missing_waits(res.stdout.splitlines())
        copies += n
        assert not bad, "%d of %d copies, the first in %s: %s before %s" % ((len(bad), n) + bad[0])
    assert copies > 1000
