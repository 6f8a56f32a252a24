"""The built gfx950 code keeps the distances that the hardware does not: a buffer instruction
may read a scalar register as descriptor or offset only five wait states after a vector
instruction wrote it (v_readlane, v_readfirstlane, compares, carries).  The compiler sees to
that for the instructions it makes itself, and not for those inside inline assembly."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from test_abi import L  # noqa: F401  (the fixture that builds the library where there is none)

WAITS = 5
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
OBJDUMP = shutil.which("llvm-objdump", path=os.pathsep.join(
    [os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin"), os.environ.get("PATH", "")]))


def code_objects(path):
    """The gfx950 ELF images inside a shared library's offload bundles."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        head = at + len(MAGIC)
        entries, = struct.unpack_from("<Q", data, head)
        head += 8
        for _ in range(entries):
            off, size, name = struct.unpack_from("<3Q", data, head)
            if b"gfx950" in data[head + 24:head + 24 + name]:
                yield data[at + off:at + off + size]
            head += 24 + name
        at = data.find(MAGIC, at + len(MAGIC))


def scalars(text):
    """Numbers of the scalar registers that an operand list names (vcc as -1)."""
    regs = {-1} if "vcc" in text else set()
    for lo, hi, one in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        regs.update(range(int(lo), int(hi) + 1) if lo else [int(one)])
    return regs


def vector_writes(op, operands):
    """Scalar registers that a vector instruction writes."""
    if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
        return scalars(operands[0])
    if "_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")):
        return scalars(operands[1]) if len(operands) > 1 else set()
    return set()


def too_close(listing):
    """(function, instruction) of every buffer instruction that comes too soon; how many were read."""
    bad, seen, function, last = [], 0, "", {}
    now = 0                                     # wait states passed; last: when a register was written
    for line in listing.splitlines():
        m = re.match(r"[0-9a-f]+ <(.*)>:$", line)
        if m:
            function, last, now = m.group(1), {}, now + WAITS
            continue
        if not line.startswith("\t"):
            continue
        op, _, rest = line.split("//")[0].strip().partition(" ")
        operands = rest.split(", ")
        if op.startswith("buffer_"):
            seen += 1
            if any(now - last.get(r, -WAITS) < WAITS for r in scalars(rest)):
                bad.append((function, line.split("//")[0].strip()))
        now += int(rest, 0) + 1 if op == "s_nop" else 1
        if op.startswith("v_"):
            last.update(dict.fromkeys(vector_writes(op, operands), now))
        elif op.startswith("s_"):               # a scalar write in between is waited for
            for r in scalars(operands[0]):
                last.pop(r, None)
    return bad, seen


def test_the_reader_counts_wait_states():
    def listing(*lines):
        return "0000 <f>:\n" + "".join(f"\t{x} // 0\n" for x in lines)
    load = "buffer_load_dwordx4 v0, s[48:51], s43 offen lds"
    read = "v_readlane_b32 s43, v149, 21"
    assert len(too_close(listing(read, "s_mov_b32 m0, s42", "s_nop 0", load))[0]) == 1
    assert not too_close(listing(read, "s_mov_b32 m0, s42", "s_nop 3", load))[0]
    assert not too_close(listing(read, "s_nop 4", load))[0]
    assert len(too_close(listing(read, "s_nop 3", load))[0]) == 1
    assert len(too_close(listing("v_readfirstlane_b32 s50, v1", load))[0]) == 1
    assert not too_close(listing(read, "s_mov_b32 s43, 0", load))[0]
    assert not too_close(listing("v_readlane_b32 s44, v1, 0", load))[0]


@pytest.mark.skipif(OBJDUMP is None, reason="llvm-objdump is not installed")
def test_buffer_instructions_wait_for_their_scalars(L, tmp_path):  # noqa: F811
    bad, seen = [], 0
    for i, image in enumerate(code_objects(L.library_path())):
        path = tmp_path / f"{i}.co"
        path.write_bytes(image)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True,
                              text=True, check=True).stdout
        b, n = too_close(text)
        bad, seen = bad + b, seen + n
    assert seen > 400, seen                     # the loads into LDS among them
    assert not bad, (len(bad), bad[:5])
